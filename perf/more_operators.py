"""A prompt's way through the paged 8-bit cache, as it is measured: the
rotation of queries and keys at their positions, the attention of a chunk of
new rows over the cached prefix and themselves, and the draw of the next token
from truncated logits, each in its plain form (elementary torch operations)
and, where ``own`` is true, through the library's calls.

A cache page holds ``P`` tokens of every KV head as 8-bit floats with one fp32
scale per page and head; ``block_table[b, j]`` is the page of tokens
``j * P .. j * P + P - 1`` of sequence ``b``.  The new rows of a batch lie one
sequence behind the other, those of sequence ``b`` from ``row_start[b]`` on.
"""
import math

import torch

own = False

F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TOP_EXP = {"e4m3": 9, "e5m2": 16}  # the format's largest value is 0.875 * 2^TOP_EXP (448, 57344)
TYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    attn = dict(op="attention", rows="same", ragged=False, dtype="bf16", fmt="e4m3", P=64, d=128)
    rot = dict(op="rotary", d=128, rot=128, layout="half", dtype="bf16", scaling="none", theta=10000.0, pad=False)
    draw_ = dict(op="sample", settings="one", truncated=False, T=1.0, top_k=0, top_p=1.0, min_p=0.0)
    return [
        # a short turn of a conversation at the 7B shape: the smallest call, where latency counts
        dict(attn, name="chunk 7B b1 n64 l1024", B=1, N=64, Hq=32, Hkv=32, L=1024),
        # an odd-sized piece of a prompt at the 13B shape on small pages
        dict(attn, name="chunk 13B b1 n511 l4096", B=1, N=511, Hq=40, Hkv=40, L=4096, P=16),
        # prompts of every length that start without a prefix
        dict(attn, name="prompts 7B b4 n2048", B=4, N=2048, Hq=32, Hkv=32, L=0, rows="ragged"),
        # a long prompt's second piece with eight query heads to a KV head: arithmetic dominates
        dict(attn, name="chunk 70B b1 n2048 l8192", B=1, N=2048, Hq=64, Hkv=8, L=8192, P=128),
        # a running server's batch: most requests decode one token, two bring a piece of their prompt
        dict(attn, name="mixed 7B b16 l8192", B=16, N=256, Hq=32, Hkv=32, L=8192, rows="mixed", ragged=True),
        # the tiny fp32 workload, in the other 8-bit format
        dict(attn, name="chunk tiny f32 e5m2", B=2, N=40, Hq=4, Hkv=4, L=128, d=64, P=16, dtype="f32", fmt="e5m2"),
        # the rows of one verification step's tree
        dict(rot, name="rotary tree 7B b1", B=1, N=61, Hq=32, Hkv=32, L=1024),
        # pieces of long prompts, positions far past the trained length
        dict(rot, name="rotary 70B b4 n2048 far", B=4, N=2048, Hq=64, Hkv=8, L=120000, scaling="yarn"),
        # half of each head, neighbouring dims paired, fp32, a padded batch
        dict(rot, name="rotary 13B b3 part f32", B=3, N=501, Hq=40, Hkv=40, L=4096, rot=64, layout="pairs", dtype="f32",
             scaling="linear", pad=True),
        # one request's next token
        dict(draw_, name="sample 7B b1", B=1, V=32000, T=0.8, top_k=50, top_p=0.95),
        # the target rows of four trees, truncated for the acceptance that follows
        dict(draw_, name="truncate trees 7B b4", B=4 * 61, V=32000, T=0.7, top_p=0.9, truncated=True),
        # a large batch over an odd-sized vocabulary, every request with settings of its own
        dict(draw_, name="sample b128 v100003", B=128, V=100003, settings="own"),
    ]


def draw(rng):
    """One more case of the listed ranges; sizes are spread over their logarithms."""
    def log_int(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))
    pick = rng.random()
    if pick < 0.25:
        d = rng.choice([64, 128, 128])
        Hq, Hkv = rng.choice([(32, 32), (40, 40), (64, 8), (4, 4), (28, 4), (16, 1)])
        return dict(op="rotary", B=log_int(1, 16), N=log_int(1, 512), Hq=Hq, Hkv=Hkv, d=d,
                    rot=rng.choice([d, d, d // 2, 32]), layout=rng.choice(["half", "pairs"]),
                    dtype=rng.choice(["bf16", "bf16", "f32"]), scaling=rng.choice(["none", "linear", "yarn"]),
                    theta=rng.choice([10000.0, 500000.0]), L=log_int(1, 200000), pad=rng.random() < 0.3)
    if pick < 0.55:
        V = log_int(100, 131072)
        return dict(op="sample", B=log_int(1, min(256, 12800000 // V)), V=V, settings=rng.choice(["one", "own"]),
                    truncated=rng.random() < 0.3, T=rng.choice([0.0, 0.5, 0.8, 1.0, 1.3]),
                    top_k=rng.choice([0, 1, log_int(2, 200), log_int(2, 20000)]), top_p=rng.choice([1.0, 0.5, 0.9, 0.99]),
                    min_p=rng.choice([0.0, 0.0, 0.02, 0.2]))
    P, fmt = rng.choice([16, 32, 48, 64, 128]), rng.choice(["e4m3", "e4m3", "e5m2"])
    rows = rng.choice(["same", "ragged", "mixed"])
    if rng.random() < 0.15:
        return dict(op="attention", rows=rows, ragged=rng.random() < 0.5, dtype="f32", fmt=fmt, P=P,
                    d=rng.choice([64, 128]), B=log_int(1, 3), N=log_int(1, 200), Hq=8, Hkv=rng.choice([2, 4, 8]),
                    L=rng.choice([0, log_int(1, 600)]))
    Hq, Hkv = rng.choice([(32, 32), (40, 40), (64, 8), (4, 4), (28, 4), (16, 1)])
    case = dict(op="attention", rows=rows, ragged=rng.random() < 0.5, dtype="bf16", fmt=fmt, P=P,
                d=rng.choice([64, 128, 128]), B=log_int(1, 16), N=log_int(1, 2048), Hq=Hq, Hkv=Hkv,
                L=rng.choice([0, log_int(1, 8192), log_int(64, 8192), log_int(64, 8192)]))
    # the plain form holds every score of the padded batch
    while case["B"] * case["N"] * Hq * (case["L"] + case["N"] + 2 * P) > 1.3e9:
        k = "B" if case["B"] > 1 and rng.random() < 0.5 else "N" if case["N"] > case["L"] else "L"
        case[k] = max(1, case[k] * 3 // 4)
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def spread(lo, hi, n):
    """n sizes from lo to hi, in no order."""
    return [lo + (hi - lo) * ((7919 * (b + 1)) % 1009) // 1008 for b in range(n)]


def row_counts(case):
    """New rows of each sequence: part of the case's shape, so that work() knows them."""
    B, N = case["B"], case["N"]
    if case["rows"] == "same":
        return [N] * B
    if case["rows"] == "ragged":
        return [N] + spread(1, N, B - 1)
    return [N if b % 8 == 3 or B == 1 else 1 for b in range(B)]


def prefix_lengths(case):
    if not case["ragged"]:
        return [case["L"]] * case["B"]
    return spread(min(case["L"], case["L"] // 16), case["L"], case["B"])


def make_pages(gen, pages, fill, Hkv, P, d, fmt):
    """Quantised N(0, sigma^2) data, sigma per (page, head); slots past `fill` tokens hold stale bytes, NaN codes too."""
    sigma = torch.exp(0.5 * torch.randn(pages, Hkv, 1, 1, generator=gen, device="cuda"))
    x = torch.randn(pages, Hkv, P, d, generator=gen, device="cuda") * sigma
    m, e = torch.frexp(x.abs().amax(dim=(2, 3)))
    scale = torch.ldexp(torch.ones_like(m), e - TOP_EXP[fmt] + (m > 0.875))
    codes = (x / scale[:, :, None, None]).to(F8[fmt]).view(torch.uint8)
    stale = torch.randint(0, 256, (pages, 1, P, d), generator=gen, device="cuda", dtype=torch.int32).to(torch.uint8)
    past = torch.arange(P, device="cuda")[None, :] >= fill[:, None]
    codes = torch.where(past[:, None, :, None], stale, codes)
    return codes.view(F8[fmt]).contiguous(), scale.contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 1000003 + 12345)
    if case["op"] == "rotary":
        return prepare_rotary(case, gen)
    return prepare_attention(case, gen) if case["op"] == "attention" else prepare_sample(case, gen)


def prepare_attention(case, gen):
    B, Hq, Hkv, P, d, dt = case["B"], case["Hq"], case["Hkv"], case["P"], case["d"], TYPE[case["dtype"]]
    counts, lens = row_counts(case), torch.tensor(prefix_lengths(case), device="cuda")
    start = torch.tensor([0] + counts, device="cuda").cumsum(0)
    cols = max(1, -(-case["L"] // P))
    blocks = (lens + P - 1) // P
    pages = sum(-(-n // P) for n in prefix_lengths(case)) + 1
    order = torch.randperm(pages, generator=gen, device="cuda")
    first = torch.cumsum(blocks, 0) - blocks
    col = torch.arange(cols, device="cuda")
    live = col[None, :] < blocks[:, None]
    place = order[(first[:, None] + col[None, :]).clamp(max=pages - 1)]
    table = torch.where(live, place, -1).to(torch.int32).contiguous()
    fill = torch.zeros(pages + 1, dtype=torch.int64, device="cuda")
    held = (lens[:, None] - col[None, :] * P).clamp(0, P)
    fill.scatter_(0, torch.where(live, place, pages).reshape(-1), torch.where(live, held, 0).reshape(-1))
    k_pages, k_scale = make_pages(gen, pages, fill[:pages], Hkv, P, d, case["fmt"])
    v_pages, v_scale = make_pages(gen, pages, fill[:pages], Hkv, P, d, case["fmt"])
    T = sum(counts)
    qkv = torch.randn(T, Hq + 2 * Hkv, d, generator=gen, device="cuda").to(dt)  # what one projection writes
    return dict(case=dict(case), k_pages=k_pages, v_pages=v_pages, k_scale=k_scale, v_scale=v_scale, block_table=table,
                prefix_len=lens.to(torch.int32), row_start=start.to(torch.int32).contiguous(),
                q=qkv[:, :Hq].contiguous(), k_new=qkv[:, Hq:Hq + Hkv].contiguous(), v_new=qkv[:, Hq + Hkv:],
                out=torch.zeros(T, Hq, d, dtype=dt, device="cuda"), lse=torch.zeros(T, Hq, device="cuda"))


def frequencies(case):
    """Angle per position of each pair of dims, and the factor on the rotated values."""
    n, theta = case["rot"] // 2, case["theta"]
    f = theta ** (-torch.arange(n, dtype=torch.float64) / n)
    if case["scaling"] == "none":
        return f, 1.0
    if case["scaling"] == "linear":
        return f / 4, 1.0
    # dims that turn more than 32 times over 4096 tokens stay, those that turn less than once are slowed down 32 times
    at = n * torch.log(4096 / (torch.tensor([32.0, 1.0], dtype=torch.float64) * 2 * math.pi)) / math.log(theta)
    lo, hi = max(0.0, float(at[0].floor())), min(n - 1.0, float(at[1].ceil()))
    keep = 1 - ((torch.arange(n, dtype=torch.float64) - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
    return f * keep + f / 32 * (1 - keep), 0.1 * math.log(32) + 1


def prepare_rotary(case, gen):
    B, N, Hq, Hkv, d, dt = case["B"], case["N"], case["Hq"], case["Hkv"], case["d"], TYPE[case["dtype"]]
    T = B * N
    qkv = torch.randn(T, Hq + 2 * Hkv, d, generator=gen, device="cuda").to(dt)
    first = torch.randint(case["L"] // 2, case["L"] + 1, (B, 1), generator=gen, device="cuda")
    at = first + torch.arange(N, device="cuda")
    if case["pad"]:  # rows of a padded batch that hold no token
        held = torch.randint(1, N + 1, (B, 1), generator=gen, device="cuda")
        at = torch.where(torch.arange(N, device="cuda") < held, at, -1)
    f, factor = frequencies(case)
    return dict(case=dict(case), q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], positions=at.reshape(-1).to(torch.int32),
                freq=f.to("cuda"), factor=factor, q_out=torch.zeros(T, Hq, d, dtype=dt, device="cuda"),
                k_out=torch.zeros(T, Hkv, d, dtype=dt, device="cuda"))


def prepare_sample(case, gen):
    B, V = case["B"], case["V"]
    rank = torch.argsort(torch.rand(B, V, generator=gen, device="cuda"), 1)  # logits fall with a token's rank
    z = -1.2 * torch.log(rank + 1.0) + torch.randn(B, V, generator=gen, device="cuda")
    pick = lambda *x: torch.tensor(x, device="cuda")[torch.randint(0, len(x), (B,), generator=gen, device="cuda")]  # noqa: E731
    if case["settings"] == "own":
        T, top_k = pick(0.0, 0.6, 0.8, 1.0, 1.0, 1.4), pick(0, 0, 1, 20, 50, 1000).to(torch.int32)
        top_p, min_p = pick(1.0, 1.0, 0.5, 0.9, 0.95, 0.999), pick(0.0, 0.0, 0.05, 0.1)
    else:
        fill = lambda x, t: torch.full((B,), x, dtype=t, device="cuda")  # noqa: E731
        T, top_k = fill(case["T"], torch.float32), fill(min(case["top_k"], V), torch.int32)
        top_p, min_p = fill(case["top_p"], torch.float32), fill(case["min_p"], torch.float32)
    return dict(case=dict(case), logits=z.contiguous(), temperature=T, top_k=top_k, top_p=top_p, min_p=min_p,
                uniforms=torch.rand(B, generator=gen, device="cuda"), token=torch.zeros(B, dtype=torch.int32, device="cuda"),
                logprob=torch.zeros(B, device="cuda"),
                truncated=torch.zeros(B, V, device="cuda") if case["truncated"] else None)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    if own:
        return run_own(state)
    op = state["case"]["op"]
    if op == "attention":
        return plain_attention(state)
    return plain_rotary(state) if op == "rotary" else plain_sample(state)


def run_own(s):
    import speculative_decoding_eagle_gb300.binding as E
    case = s["case"]
    dt = E.ET_F32 if case.get("dtype") == "f32" else E.ET_BF16
    if case["op"] == "attention":
        if "plan" not in s:  # what a program makes once: the shape, the cache's handle, the workspace
            s["cache"] = E.PagedCache(s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"])
            s["plan"] = E.ChunkAttnShape(B=case["B"], rows=s["q"].shape[0], Hq=case["Hq"], max_rows=case["N"], dtype=dt,
                                         max_blocks=s["block_table"].shape[1], max_prefix=case["L"])
            s["ws"] = E.new_workspace(E.et_chunk_attention_paged_workspace_size(s["plan"], s["cache"]))
        E.et_chunk_attention_paged(s["plan"], s["cache"], s["block_table"], s["prefix_len"], s["row_start"], s["q"],
                                   s["k_new"], s["v_new"], s["out"], lse=s["lse"], ws=s["ws"])
        return dict(out=s["out"], lse=s["lse"])
    if case["op"] == "rotary":
        if "plan" not in s:
            s["plan"] = E.RotaryShape(rows=s["q"].shape[0], Hq=case["Hq"], Hkv=case["Hkv"], d=case["d"], rot=case["rot"],
                                      layout=E.ET_ROTARY_HALF if case["layout"] == "half" else E.ET_ROTARY_PAIRS,
                                      dtype=dt, factor=s["factor"])
        E.et_rotary(s["plan"], s["positions"], s["freq"], s["q"], s["q_out"], k=s["k"], k_out=s["k_out"])
        return dict(q=s["q_out"], k=s["k_out"])
    E.et_sample(s["logits"], s["uniforms"], s["token"], temperature=s["temperature"], top_k=s["top_k"],
                top_p=s["top_p"], min_p=s["min_p"], logprob=s["logprob"], truncated=s["truncated"])
    return sample_outputs(s)


def sample_outputs(s):
    o = dict(token=s["token"], logprob=s["logprob"])
    return dict(o, truncated=s["truncated"]) if s["truncated"] is not None else o


def plain_attention(s):
    """The batch padded to its longest sequence; every score held at once."""
    case = s["case"]
    B, N, Hq, Hkv, P, d = (case[k] for k in ("B", "N", "Hq", "Hkv", "P", "d"))
    G, cols, T = Hq // Hkv, s["block_table"].shape[1], s["q"].shape[0]
    L = cols * P
    table = s["block_table"].long().clamp(min=0)
    start = s["row_start"].long()
    i = torch.arange(N, device="cuda")
    there = i[None, :] < (start[1:] - start[:-1])[:, None]                     # [B, N]
    row = (start[:-1, None] + i[None, :]).clamp(max=T - 1)
    inside = torch.arange(L, device="cuda")[None, :] < s["prefix_len"][:, None]
    live = torch.cat([inside, there], 1)                                       # [B, L + N] keys that exist

    def rows(pages, scale, new):
        x = pages.view(torch.uint8)[table].view(pages.dtype).float() * scale[table][..., None, None]
        x = x.permute(0, 2, 1, 3, 4).reshape(B, Hkv, L, d)
        x = torch.cat([x, new[row].float().permute(0, 2, 1, 3)], 2)
        return torch.where(live[:, None, :, None], x, 0)                       # stale slots are never read
    k, v = rows(s["k_pages"], s["k_scale"], s["k_new"]), rows(s["v_pages"], s["v_scale"], s["v_new"])
    q = s["q"][row].float().view(B, N, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, N * G, d)
    z = torch.matmul(q, k.transpose(2, 3)).mul_(d ** -0.5).view(B, Hkv, N, G, L + N)
    sees = torch.cat([inside[:, None, :].expand(B, N, L), there[:, None, :] & (i[None, None, :] <= i[None, :, None])], 2)
    z.masked_fill_(~sees[:, None, :, None, :], float("-inf"))
    top = z.amax(-1, keepdim=True)
    p = z.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.div_(total).view(B, Hkv, N * G, L + N), v).view(B, Hkv, N, G, d)
    s["out"].copy_(out.permute(0, 2, 1, 3, 4).reshape(B, N, Hq, d)[there])
    s["lse"].copy_((top + torch.log(total))[..., 0].permute(0, 2, 1, 3).reshape(B, N, Hq)[there])
    return dict(out=s["out"], lse=s["lse"])


def plain_rotary(s):
    case = s["case"]
    rot, half = case["rot"], case["layout"] == "half"
    angle = s["positions"].double()[:, None] * s["freq"]                       # far positions: in 64 bits
    c = (torch.cos(angle) * s["factor"]).float()[:, None]
    d = (torch.sin(angle) * s["factor"]).float()[:, None]
    there = (s["positions"] >= 0)[:, None, None]
    for x, out in ((s["q"], s["q_out"]), (s["k"], s["k_out"])):
        t = x[..., :rot].float()
        a, b = (t[..., :rot // 2], t[..., rot // 2:]) if half else (t[..., 0::2], t[..., 1::2])
        u, w = a * c - b * d, a * d + b * c
        turned = torch.cat([u, w], -1) if half else torch.stack([u, w], -1).flatten(-2)
        out.copy_(torch.where(there, torch.cat([turned, x[..., rot:].float()], -1).to(x.dtype), out))
    return dict(q=s["q_out"], k=s["k_out"])


def plain_sample(s):
    """Tokens in the order of their logits; masses in 64 bits, since a token next to a border goes one way or the other."""
    z, T = s["logits"], s["temperature"].double()[:, None]
    V = z.shape[1]
    greedy = T == 0
    z_sorted, order = torch.sort(z, dim=1, descending=True, stable=True)
    depth = (z_sorted - z_sorted[:, :1].double()) / torch.where(greedy, 1.0, T)  # log of the weight relative to the top
    k = torch.where(greedy[:, 0], 1, torch.where(s["top_k"] > 0, s["top_k"].long(), V))[:, None]
    w = torch.exp(depth) * (torch.arange(V, device="cuda")[None, :] < k)
    before = torch.cumsum(w, 1) - w
    p, m = s["top_p"].double()[:, None], s["min_p"].double()[:, None]
    keep = (w > 0) & ((p >= 1) | (before < p * w.sum(1, keepdim=True)))
    keep &= (m <= 0) | (depth >= torch.log(m))
    keep[:, 0] = True
    w = torch.zeros_like(w).scatter_(1, order, torch.where(keep, w, 0))         # back in the order of ids
    mass = torch.cumsum(w, 1)
    total = mass[:, -1:]
    s["token"].copy_((mass <= s["uniforms"].double()[:, None] * total).sum(1))
    s["logprob"].copy_(torch.log(torch.gather(w, 1, s["token"].long()[:, None]) / total)[:, 0])
    if s["truncated"] is not None:
        s["truncated"].copy_(torch.where(w > 0, z, float("-inf")))
    return sample_outputs(s)


# ---------------------------------------------------------------------------
# work and the value in 64 bits
# ---------------------------------------------------------------------------
def work(case):
    if case["op"] == "sample":
        B, V = case["B"], case["V"]
        return dict(bytes=4 * B * V * (2 if case["truncated"] else 1) + 28 * B, flops=0)
    es, d, Hq, Hkv = (2 if case["dtype"] == "bf16" else 4), case["d"], case["Hq"], case["Hkv"]
    if case["op"] == "rotary":
        T = case["B"] * case["N"]
        return dict(bytes=T * (2 * (Hq + Hkv) * d * es + 4), flops=0)
    n, lens = row_counts(case), prefix_lengths(case)
    T, tokens, pages = sum(n), sum(lens), sum(-(-x // case["P"]) for x in lens)
    bytes_ = 2 * Hkv * d * tokens + 8 * Hkv * pages + 4 * pages
    bytes_ += 2 * T * Hkv * d * es + 2 * T * Hq * d * es + 4 * T * Hq
    return dict(bytes=bytes_, flops=4.0 * Hq * d * sum(x * y + x * (x + 1) / 2 for x, y in zip(n, lens)))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attention":
        return exact_attention(s)
    return exact_rotary(s) if case["op"] == "rotary" else exact_sample(s)


def exact_attention(s):
    """Sequence by sequence and KV head by KV head, over the tokens that are there."""
    case = s["case"]
    Hq, Hkv, P, d = (case[k] for k in ("Hq", "Hkv", "P", "d"))
    G = Hq // Hkv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    for b in range(case["B"]):
        n, r0, r1 = int(s["prefix_len"][b]), int(s["row_start"][b]), int(s["row_start"][b + 1])
        pages = s["block_table"][b, :-(-n // P)].long()
        own_part = torch.ones(r1 - r0, r1 - r0, dtype=torch.bool, device="cuda").tril()
        sees = torch.cat([torch.ones(r1 - r0, n, dtype=torch.bool, device="cuda"), own_part], 1)
        for g in range(Hkv):
            def column(codes, scale, new):
                held = codes.view(torch.uint8)[pages, g].view(codes.dtype).double() * scale[pages, g].double()[:, None, None]
                return torch.cat([held.reshape(-1, d)[:n], new[r0:r1, g].double()])
            k, v = column(s["k_pages"], s["k_scale"], s["k_new"]), column(s["v_pages"], s["v_scale"], s["v_new"])
            q = s["q"][r0:r1, g * G:(g + 1) * G].double()
            z = torch.einsum("nhd,td->hnt", q, k) / math.sqrt(d)
            z = torch.where(sees[None], z, -math.inf)
            total = torch.logsumexp(z, -1)
            out[r0:r1, g * G:(g + 1) * G] = torch.einsum("hnt,td->nhd", torch.exp(z - total[..., None]), v)
            lse[r0:r1, g * G:(g + 1) * G] = total.T
    return dict(out=out, lse=lse)


def exact_rotary(s):
    """Pairs of dims as complex numbers, turned by a complex factor."""
    case = s["case"]
    rot, pos = case["rot"], s["positions"]
    turn = torch.polar(torch.full((len(pos), rot // 2), s["factor"], dtype=torch.float64, device="cuda"),
                       torch.outer(pos.double(), s["freq"]))[:, None]
    o = {}
    for name in ("q", "k"):
        x = s[name].double()
        y = torch.zeros_like(x)
        if case["layout"] == "half":
            w = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * turn
            y[..., :rot // 2], y[..., rot // 2:rot] = w.real, w.imag
        else:
            w = torch.view_as_complex(x[..., :rot].contiguous().unflatten(-1, (-1, 2))) * turn
            y[..., :rot] = torch.view_as_real(w).flatten(-2)
        y[..., rot:] = x[..., rot:]
        y[pos < 0] = 0  # left as it was
        o[name] = y
    return o


def exact_sample(s):
    """Row by row: the kept tokens from the definition, then the log-probability of the token that is drawn from them."""
    B, V = s["logits"].shape
    logprob = torch.zeros(B, dtype=torch.float64, device="cuda")
    truncated = torch.full((B, V), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(B):
        z = s["logits"][b].double()
        T, k, p, m = (float(s[n][b]) for n in ("temperature", "top_k", "top_p", "min_p"))
        ids = torch.argsort(-z, dim=0, stable=True)
        if T == 0:
            kept = ids[:1]
            q = torch.zeros(V, dtype=torch.float64, device="cuda")
        else:
            kept = ids[:int(k)] if k > 0 else ids
            q = (z - z.max()) / T
            if p < 1:
                share = torch.softmax(q[kept], 0)
                need = int(torch.searchsorted(torch.cumsum(share, 0), torch.tensor(p, dtype=torch.float64, device="cuda"))) + 1
                kept = kept[:need]
            if m > 0:
                kept = kept[(q[kept] >= math.log(m)) | (kept == ids[0])]
        kept = torch.sort(kept)[0]
        share = torch.softmax(q[kept], 0)
        at = int((torch.cumsum(share, 0) <= float(s["uniforms"][b])).sum())
        logprob[b] = torch.log(share[min(at, len(kept) - 1)])
        truncated[b, kept] = z[kept]
    o = dict(token=None, logprob=logprob)
    return dict(o, truncated=truncated) if s["truncated"] is not None else o
