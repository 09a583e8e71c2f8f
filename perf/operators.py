"""The paged 8-bit KV cache of the verification step, as it is measured: the
attention that reads it, the commit that writes it and the block map that
lays it out, each in its plain form (elementary torch operations) and, where
``own`` is true, through the library's calls.

A cache page holds ``P`` tokens of every KV head as 8-bit floats with one fp32
scale per page and head; ``block_table[b, j]`` is the page of tokens
``j * P .. j * P + P - 1`` of sequence ``b``.
"""
import math

import torch

own = False

F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TOP_EXP = {"e4m3": 9, "e5m2": 16}  # the format's largest value is 0.875 * 2^TOP_EXP (448, 57344)
EXP_MIN, EXP_MAX = -48, 48         # range of a page scale's exponent


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    attn = dict(op="attention", ragged=False, dtype="bf16", fmt="e4m3", P=64, d=128)
    commit = dict(op="commit", fmt="e4m3", P=64, d=128, dtype="bf16")
    return [
        # one request decoding one token: the smallest serving call, where latency counts
        dict(attn, name="decode 7B b1 l1023", B=1, N=1, Hq=32, Hkv=32, L=1023),
        # a batch of requests of every length decoding one token each, eight query heads to a KV head
        dict(attn, name="decode 70B b16 ragged", B=16, N=1, Hq=64, Hkv=8, L=16384, ragged=True),
        # the verification step's tree of 61 rows at the 7B shape
        dict(attn, name="tree 7B b1 l1024", B=1, N=61, Hq=32, Hkv=32, L=1024),
        # the 13B shape on small pages
        dict(attn, name="tree 13B b1 l4096", B=1, N=61, Hq=40, Hkv=40, L=4096, P=16),
        # grouped heads: 648 query rows share each KV head, so arithmetic dominates
        dict(attn, name="tree 70B b1 l8192", B=1, N=81, Hq=64, Hkv=8, L=8192, P=128),
        # the batched sweep: trees of 16 sequences over prefixes of every length
        dict(attn, name="tree 7B b16 ragged", B=16, N=61, Hq=32, Hkv=32, L=16384, ragged=True),
        # the tiny fp32 workload, in the other 8-bit format
        dict(attn, name="tree tiny f32 e5m2", B=1, N=17, Hq=4, Hkv=4, L=128, d=64, P=16, dtype="f32", fmt="e5m2"),
        # what one verified step appends: a path of up to 7 rows, with the features of the rows
        dict(commit, name="commit 7B b1", B=1, N=61, Hkv=32, path_len=7, L=1021, F=4096),
        # the same for a batch, no features
        dict(commit, name="commit 7B b32", B=32, N=61, Hkv=32, path_len=7, L=2048, F=0),
        # a prompt written into the cache behind an earlier, odd-sized part
        dict(commit, name="prompt 7B b2 x 2047", B=2, N=2047, Hkv=32, path_len=0, L=77, F=0),
        # two scheduler steps of a running batch: lengths move on, some requests end and others start
        dict(op="map", name="block map b32", B=32, P=64, L=16384, max_new=61),
        # the same for a large server
        dict(op="map", name="block map b1024", B=1024, P=16, L=8192, max_new=128),
    ]


def draw(rng):
    """One more case of the listed ranges; sizes are spread over their logarithms."""
    def log_int(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))
    P = rng.choice([16, 32, 48, 64, 128])
    fmt = rng.choice(["e4m3", "e4m3", "e5m2"])
    pick = rng.random()
    if pick < 0.2:
        return dict(op="map", B=log_int(1, 1024), P=P, L=log_int(64, 8192), max_new=log_int(1, 128))
    if pick < 0.45:
        prompt = rng.random() < 0.4
        N = log_int(64, 2047) if prompt else log_int(2, 128)
        return dict(op="commit", fmt=fmt, P=P, d=rng.choice([64, 128]), dtype=rng.choice(["bf16", "bf16", "f32"]),
                    B=log_int(1, 4 if prompt else 32), N=N,
                    Hkv=rng.choice([4, 8, 32, 40]), path_len=0 if prompt else min(N, rng.randint(2, 17)),
                    L=log_int(1, 2048), F=0 if prompt else rng.choice([0, 512, 4096]))
    f32 = rng.random() < 0.15
    if f32:
        return dict(op="attention", ragged=rng.random() < 0.5, dtype="f32", fmt=fmt, P=P, d=rng.choice([64, 128]),
                    B=log_int(1, 3), N=log_int(1, 40), Hq=8, Hkv=rng.choice([2, 4, 8]), L=log_int(2, 600))
    Hq, Hkv = rng.choice([(32, 32), (40, 40), (64, 8), (4, 4), (28, 4), (16, 1)])
    case = dict(op="attention", ragged=rng.random() < 0.5, dtype="bf16", fmt=fmt, P=P, d=rng.choice([64, 128, 128]),
                B=log_int(1, 16), N=1 if rng.random() < 0.4 else log_int(2, 128), Hq=Hq, Hkv=Hkv, L=log_int(2, 16384))
    while work(case)["flops"] > 3e10 and case["L"] > 64:
        case["L"] = case["L"] * 3 // 4
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def lengths(case):
    """Prefix lengths of an attention case: part of its shape, so that work() knows them."""
    if not case["ragged"]:
        return [case["L"]] * case["B"]
    lo, hi = min(512, max(1, case["L"] // 8)), case["L"]
    return [lo + (hi - lo) * ((7919 * (b + 1)) % 1009) // 1008 for b in range(case["B"])]


def make_pages(gen, pages, fill, Hkv, P, d, fmt):
    """Quantised N(0, sigma^2) data, sigma per (page, head); slots past `fill` tokens hold stale bytes, NaN codes too."""
    sigma = torch.exp(0.5 * torch.randn(pages, Hkv, 1, 1, generator=gen, device="cuda"))
    x = torch.randn(pages, Hkv, P, d, generator=gen, device="cuda") * sigma
    m, e = torch.frexp(x.abs().amax(dim=(2, 3)))
    k = (e - TOP_EXP[fmt] + (m > 0.875)).clamp(EXP_MIN, EXP_MAX)
    scale = torch.ldexp(torch.ones_like(m), k)
    codes = (x / scale[:, :, None, None]).to(F8[fmt]).view(torch.uint8)
    stale = torch.randint(0, 256, (pages, 1, P, d), generator=gen, device="cuda", dtype=torch.int32).to(torch.uint8)
    past = torch.arange(P, device="cuda")[None, :] >= fill[:, None]
    codes = torch.where(past[:, None, :, None], stale, codes)
    return codes.view(F8[fmt]).contiguous(), scale.contiguous()


def tree_mask(gen, B, N):
    """Ancestor bitmask (uint64 words in int64) of random trees whose row 0 is the root."""
    bits = torch.zeros(B, N, N, dtype=torch.bool, device="cuda")
    bits[:, 0, 0] = True
    at = torch.arange(B, device="cuda")
    u = torch.rand(B, N, generator=gen, device="cuda")
    for i in range(1, N):
        parent = (u[:, i] * min(i, 40)).long() + max(0, i - 40)
        bits[:, i] = bits[at, parent]
        bits[:, i, i] = True
    W = (N + 63) // 64
    padded = torch.zeros(B, N, W * 64, dtype=torch.int64, device="cuda")
    padded[:, :, :N] = bits
    words = (padded.view(B, N, W, 64) << torch.arange(64, device="cuda")).sum(-1)
    return bits, words.contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 1000003 + 12345)
    if case["op"] == "map":
        return prepare_map(case, gen)
    B, Hkv, P, d, fmt = case["B"], case["Hkv"], case["P"], case["d"], case["fmt"]
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    randn = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(dt)  # noqa: E731
    if case["op"] == "attention":
        lens = torch.tensor(lengths(case), device="cuda")
        room = case["L"]
    else:
        lo = max(0, case["L"] // 2) if B > 1 else case["L"]
        lens = torch.randint(lo, case["L"] + 1, (B,), generator=gen, device="cuda")
        room = case["L"] + (case["path_len"] or case["N"])
    cols = max(1, -(-room // P))
    blocks = (lens + (0 if case["op"] == "attention" else case["path_len"] or case["N"]) + P - 1) // P
    first = torch.cumsum(blocks, 0) - blocks
    col = torch.arange(cols, device="cuda")
    live = col[None, :] < blocks[:, None]
    pages = sum(-(-n // P) for n in lengths(case)) if case["op"] == "attention" else B * cols
    order = torch.randperm(pages + 1, generator=gen, device="cuda")  # page order[pages] belongs to nobody
    place = (first[:, None] + col[None, :]).clamp(max=max(pages, 1) - 1)
    table = torch.where(live, order[place], -1).to(torch.int32).contiguous()
    fill = torch.zeros(pages + 1, dtype=torch.int64, device="cuda")
    held = (lens[:, None] - col[None, :] * P).clamp(0, P)
    fill.scatter_(0, torch.where(live, order[place], order[pages]).reshape(-1), torch.where(live, held, 0).reshape(-1))
    k_pages, k_scale = make_pages(gen, pages + 1, fill, Hkv, P, d, fmt)
    v_pages, v_scale = make_pages(gen, pages + 1, fill, Hkv, P, d, fmt)
    s = dict(case=dict(case), k_pages=k_pages, v_pages=v_pages, k_scale=k_scale, v_scale=v_scale, block_table=table,
             prefix_len=lens.to(torch.int32), k_tree=randn(B, case["N"], Hkv, d), v_tree=randn(B, case["N"], Hkv, d))
    if case["op"] == "attention":
        N, Hq = case["N"], case["Hq"]
        s["q"] = randn(B, N, Hq, d)
        s["bits"], s["mask"] = tree_mask(gen, B, N)
        s["out"] = torch.zeros(B, N, Hq, d, dtype=dt, device="cuda")
        s["lse"] = torch.zeros(B, Hq, N, device="cuda")
        return s
    n, F = case["path_len"] or case["N"], case["F"]
    s["spare"] = order[pages]
    if case["path_len"]:
        s["accept_len"] = torch.randint(0, n, (B,), generator=gen, device="cuda", dtype=torch.int32)
        rows = torch.sort(torch.rand(B, case["N"], generator=gen, device="cuda")[:, 1:].argsort(1)[:, :n - 1] + 1, 1)[0]
        path = torch.cat([torch.zeros(B, 1, dtype=torch.int64, device="cuda"), rows], 1)
        unused = torch.arange(n, device="cuda")[None, :] > s["accept_len"][:, None]
        s["path"] = torch.where(unused, -1, path).to(torch.int32).contiguous()
    else:
        s["accept_len"] = torch.full((B,), n - 1, dtype=torch.int32, device="cuda")
        s["path"] = None
    s["new_prefix_len"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    s["features"] = randn(B, case["N"], F) if F else None
    s["feat_out"] = torch.zeros(B, n, F, dtype=dt, device="cuda") if F else None
    return s


def prepare_map(case, gen):
    """A running batch, its blocks scattered over the pool, and the lengths of its next two steps."""
    B, P, L, M = case["B"], case["P"], case["L"], case["max_new"]
    cols = -(-(L + M) // P)
    lens = torch.randint(0, L + 1, (3, B), generator=gen, device="cuda")
    stay = torch.rand(2, B, generator=gen, device="cuda")
    a = torch.minimum(torch.where(stay[0] < 0.9, lens[0] + (stay[0] * 16).long(), lens[1]), torch.tensor(L, device="cuda"))
    b = torch.minimum(torch.where(stay[1] < 0.9, a + (stay[1] * 16).long(), lens[2]), torch.tensor(L, device="cuda"))
    a = torch.where((stay[0] > 0.9) & (stay[0] < 0.93), 0, a)  # ended: every block goes back
    new = torch.randint(1, M + 1, (2, B), generator=gen, device="cuda")
    new = torch.where(torch.stack([a, b]) == 0, 0, new)
    have = (lens[0] + P - 1) // P
    pool = B * cols  # whatever the lengths, the pool holds them
    order = torch.randperm(pool, generator=gen, device="cuda")
    first = torch.cumsum(have, 0) - have
    col = torch.arange(cols, device="cuda")
    table = torch.where(col[None, :] < have[:, None], order[(first[:, None] + col[None, :]).clamp(max=pool - 1)], -1)
    used = have.sum()
    free_list = order[(torch.arange(pool, device="cuda") + used) % pool]
    i32 = lambda t: t.to(torch.int32).contiguous()  # noqa: E731
    return dict(case=dict(case), lens=[i32(a), i32(b)], new=[i32(new[0]), i32(new[1])], n_blocks=i32(have),
                block_table=i32(table), free_list=i32(free_list), free_count=i32((pool - used).reshape(1)),
                slot_map=[torch.zeros(B, M, dtype=torch.int64, device="cuda") for _ in range(2)])


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    if own:
        return run_own(state)
    op = state["case"]["op"]
    if op == "attention":
        return plain_attention(state)
    return plain_commit(state) if op == "commit" else plain_map(state)


def run_own(s):
    import speculative_decoding_eagle_gb300.binding as E
    case = s["case"]
    if "plan" not in s:  # what a program makes once: the shape, the cache's handle, the workspace
        if case["op"] == "map":
            s["plan"] = E.BlockMapShape(B=case["B"], page_size=case["P"], max_blocks=s["block_table"].shape[1],
                                        num_pages=s["free_list"].shape[0], max_new=case["max_new"])
        else:
            dt = E.ET_BF16 if case["dtype"] == "bf16" else E.ET_F32
            s["cache"] = E.PagedCache(s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"])
            if case["op"] == "attention":
                s["plan"] = E.PagedAttnShape(B=case["B"], N=case["N"], Hq=case["Hq"], dtype=dt, max_prefix=case["L"],
                                             max_blocks=s["block_table"].shape[1])
                s["ws"] = E.new_workspace(E.et_tree_attention_paged_workspace_size(s["plan"], s["cache"]))
            else:
                s["plan"] = E.PagedCommitShape(B=case["B"], N=case["N"], path_len=case["path_len"], dtype=dt,
                                               max_blocks=s["block_table"].shape[1], feat_dim=case["F"])
    if case["op"] == "attention":
        E.et_tree_attention_paged(s["plan"], s["cache"], s["block_table"], s["prefix_len"], s["q"], s["k_tree"],
                                  s["v_tree"], s["mask"], s["out"], lse=s["lse"], ws=s["ws"])
        return dict(out=s["out"], lse=s["lse"])
    if case["op"] == "commit":
        E.et_kv_commit_paged(s["plan"], s["cache"], s["block_table"], s["k_tree"], s["v_tree"], s["accept_len"],
                             s["path"], s["prefix_len"], s["new_prefix_len"], features=s["features"],
                             feat_out=s["feat_out"])
        return commit_outputs(s)
    for step in range(2):
        E.et_block_map(s["plan"], s["lens"][step], s["new"][step], s["n_blocks"], s["block_table"], s["free_list"],
                       s["free_count"], s["slot_map"][step])
    return map_outputs(s)


def commit_outputs(s):
    o = dict(k_pages=s["k_pages"], v_pages=s["v_pages"], k_scale=s["k_scale"], v_scale=s["v_scale"],
             new_prefix_len=s["new_prefix_len"])
    return dict(o, feat_out=s["feat_out"]) if s["feat_out"] is not None else o


def map_outputs(s):
    return dict(n_blocks=s["n_blocks"], block_table=s["block_table"], free_list=s["free_list"],
                free_count=s["free_count"], slots_a=s["slot_map"][0], slots_b=s["slot_map"][1])


def plain_attention(s):
    case = s["case"]
    B, N, Hq, Hkv, P, d = (case[k] for k in ("B", "N", "Hq", "Hkv", "P", "d"))
    G, cols = Hq // Hkv, s["block_table"].shape[1]
    L = cols * P
    table = s["block_table"].long().clamp(min=0)

    def rows(pages, scale, tree):  # the sequence's tokens then its tree rows, [B, Hkv, L + N, d]
        x = pages.view(torch.uint8)[table].view(pages.dtype).float() * scale[table][..., None, None]
        x = x.permute(0, 2, 1, 3, 4).reshape(B, Hkv, L, d)
        return torch.cat([x, tree.float().permute(0, 2, 1, 3)], 2)
    inside = torch.arange(L, device="cuda")[None, :] < s["prefix_len"][:, None]
    keep = torch.cat([inside[:, None, :].expand(B, N, L), s["bits"]], 2)                     # [B, N, L + N]
    any_row = keep.any(1)                                                                    # stale slots are never read
    k = torch.where(any_row[:, None, :, None], rows(s["k_pages"], s["k_scale"], s["k_tree"]), 0)
    v = torch.where(any_row[:, None, :, None], rows(s["v_pages"], s["v_scale"], s["v_tree"]), 0)
    q = s["q"].float().view(B, N, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, N * G, d)
    z = torch.matmul(q, k.transpose(2, 3)) * d ** -0.5
    z = z.view(B, Hkv, N, G, L + N).masked_fill(~keep[:, None, :, None, :], float("-inf"))
    top = z.amax(-1, keepdim=True)
    p = torch.exp(z - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul((p / total).view(B, Hkv, N * G, L + N), v).view(B, Hkv, N, G, d)
    s["out"].copy_(out.permute(0, 2, 1, 3, 4).reshape(B, N, Hq, d))
    s["lse"].copy_((top + torch.log(total))[..., 0].permute(0, 1, 3, 2).reshape(B, Hq, N))
    return dict(out=s["out"], lse=s["lse"])


def plain_commit(s):
    case = s["case"]
    B, N, P, fmt = case["B"], case["N"], case["P"], case["fmt"]
    n = case["path_len"] or N
    touch = (n + 2 * P - 2) // P                                                    # pages a sequence may write to
    base = s["prefix_len"].long()
    cell = (base // P)[:, None] + torch.arange(touch, device="cuda")                # [B, touch] block numbers
    i = cell[:, :, None] * P + torch.arange(P, device="cuda") - base[:, None, None]  # position in the path, [B, touch, P]
    fresh = (i >= 0) & (i <= s["accept_len"][:, None, None])
    at = i.clamp(0, n - 1)
    b = torch.arange(B, device="cuda")
    path = s["path"].long() if s["path"] is not None else torch.arange(N, device="cuda").expand(B, N)
    row = path[b[:, None, None], at].clamp(min=0)
    used = fresh.any(2)
    cols = s["block_table"].shape[1]
    page = torch.where(used, s["block_table"].long()[b[:, None], cell.clamp(max=cols - 1)], s["spare"])
    begun = cell * P < base[:, None]
    for pages, scale, tree in ((s["k_pages"], s["k_scale"], s["k_tree"]), (s["v_pages"], s["v_scale"], s["v_tree"])):
        x = tree[b[:, None, None], row].float()                                     # [B, touch, P, Hkv, d]
        x = torch.where(fresh[..., None, None], x, 0).transpose(2, 3)               # [B, touch, Hkv, P, d]
        m, e = torch.frexp(x.abs().amax(dim=(3, 4)))
        k = (e - TOP_EXP[fmt] + (m > 0.875)).clamp(EXP_MIN, EXP_MAX)
        need = torch.ldexp(torch.ones_like(m), torch.where(m > 0, k, EXP_MIN))
        was = scale[page]
        now = torch.where(used[..., None], torch.where(begun[..., None], torch.maximum(was, need), need), was)
        bits = pages.view(torch.uint8)
        held = bits[page]
        moved = (held.view(pages.dtype).float() * (was / now)[..., None, None]).to(pages.dtype).view(torch.uint8)
        keeps = (begun[..., None] & (now > was))[..., None, None] & (i < 0)[:, :, None, :, None]
        code = (x / now[..., None, None]).to(pages.dtype).view(torch.uint8)
        bits[page] = torch.where(fresh[:, :, None, :, None], code, torch.where(keeps, moved, held))
        scale[page] = now
    s["new_prefix_len"].copy_(base + s["accept_len"] + 1)
    if s["feat_out"] is not None:
        take = torch.arange(n, device="cuda")
        f = s["features"][b[:, None], path.clamp(min=0)]
        s["feat_out"].copy_(torch.where((take[None, :] <= s["accept_len"][:, None])[..., None], f, 0))
    return commit_outputs(s)


def plain_map(s):
    for step in range(2):
        plain_map_step(s, s["lens"][step].long(), s["new"][step].long(), s["slot_map"][step])
    return map_outputs(s)


def plain_map_step(s, lens, new, slots):
    P, cols, pool = s["case"]["P"], s["block_table"].shape[1], s["free_list"].shape[0]
    have, table, free = s["n_blocks"].long(), s["block_table"].long(), s["free_list"].long()
    count = s["free_count"].long()[0]
    need = (lens + new + P - 1) // P
    gives = (have - need).clamp(min=0)
    wants = (need - have).clamp(min=0)
    stack_size = count + gives.sum()
    served = (wants == 0) | (torch.cumsum(wants, 0) <= stack_size)
    gets = torch.where(served, wants, 0)
    col = torch.arange(cols, device="cuda")[None, :]
    going = (col >= need[:, None]) & (col < have[:, None])
    back = count + (torch.cumsum(gives, 0) - gives)[:, None] + col - need[:, None]   # place of a returned page on the stack
    stack = torch.cat([torch.where(torch.arange(pool, device="cuda") < count, free, -1), free.new_full((1,), -1)])
    stack.scatter_(0, torch.where(going, back, pool).reshape(-1), torch.where(going, table, -1).reshape(-1))
    coming = (col >= have[:, None]) & (col < (have + gets)[:, None])
    turn = (torch.cumsum(gets, 0) - gets)[:, None] + col - have[:, None]             # the turn-th page taken from the top
    got = stack[torch.where(coming, stack_size - 1 - turn, pool)]
    table = torch.where(coming, got, torch.where(going, -1, table))
    left = stack_size - gets.sum()
    s["n_blocks"].copy_(torch.where(served, need, have))
    s["block_table"].copy_(table)
    s["free_list"].copy_(torch.where(torch.arange(pool, device="cuda") < left, stack[:pool], free))
    s["free_count"].copy_(left.reshape(1))
    k = torch.arange(slots.shape[1], device="cuda")[None, :]
    pos = lens[:, None] + k
    page = torch.gather(table, 1, (pos // P).clamp(max=cols - 1))
    slots.copy_(torch.where((k < new[:, None]) & served[:, None], page * P + pos % P, -1))


# ---------------------------------------------------------------------------
# work and the value in 64 bits
# ---------------------------------------------------------------------------
def work(case):
    B, P = case["B"], case["P"]
    if case["op"] == "map":
        # two steps: lengths, new rows and block counts read, counts and slots written; a tenth of the requests change
        # whole tables (read and written once), the others a block at times
        half = case["L"] // 2
        return dict(bytes=2 * (B * (4 + 4 + 8) + B * case["max_new"] // 2 * 8 + B // 10 * (half // P) * 8), flops=0)
    es, d, Hkv, N = (2 if case["dtype"] == "bf16" else 4), case["d"], case["Hkv"], case["N"]
    if case["op"] == "attention":
        n = lengths(case)
        tokens, Hq = sum(n), case["Hq"]
        bytes_ = 2 * Hkv * d * tokens + 2 * 4 * Hkv * sum(-(-x // P) for x in n) + 4 * sum(-(-x // P) for x in n)
        bytes_ += 2 * B * N * Hkv * d * es + 2 * B * N * Hq * d * es + B * Hq * N * 4 + B * N * ((N + 63) // 64) * 8
        return dict(bytes=bytes_, flops=4.0 * N * Hq * d * (tokens + B * (N + 1) / 2))
    n = case["path_len"] or N
    rows = B * ((n + 1) / 2 if case["path_len"] else n)
    pages = B * (1 + (n if not case["path_len"] else 0) / P)
    return dict(bytes=2 * rows * Hkv * d * (es + 1) + 2 * 8 * pages * Hkv + rows * case["F"] * es + B * n * case["F"] * es,
                flops=0)


def exact(case, seed):
    if case["op"] == "map":
        return None  # whole numbers
    s = prepare(case, seed)
    return exact_attention(s) if case["op"] == "attention" else exact_commit(s)


def exact_attention(s):
    """Sequence by sequence and KV head by KV head, over the tokens that are there."""
    case = s["case"]
    B, N, Hq, Hkv, P, d = (case[k] for k in ("B", "N", "Hq", "Hkv", "P", "d"))
    G = Hq // Hkv
    out = torch.zeros(B, N, Hq, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(B, Hq, N, dtype=torch.float64, device="cuda")
    for b in range(B):
        n = int(s["prefix_len"][b])
        pages = s["block_table"][b, :-(-n // P)].long()
        for g in range(Hkv):
            def column(codes, scale, tree):
                held = codes.view(torch.uint8)[pages, g].view(codes.dtype).double() * scale[pages, g].double()[:, None, None]
                return torch.cat([held.reshape(-1, d)[:n], tree[b, :, g].double()])
            k, v = column(s["k_pages"], s["k_scale"], s["k_tree"]), column(s["v_pages"], s["v_scale"], s["v_tree"])
            sees = torch.cat([torch.ones(N, n, dtype=torch.bool, device="cuda"), s["bits"][b]], 1)
            q = s["q"][b, :, g * G:(g + 1) * G].double()
            z = torch.einsum("nhd,td->hnt", q, k) / math.sqrt(d)
            z = torch.where(sees[None], z, -math.inf)
            total = torch.logsumexp(z, -1)
            out[b, :, g * G:(g + 1) * G] = torch.einsum("hnt,td->nhd", torch.exp(z - total[..., None]), v)
            lse[b, g * G:(g + 1) * G] = total
    return dict(out=out, lse=lse)


def exact_commit(s):
    """Page by page, in 64 bits; the code nearest to a value is looked up in the list of the format's values."""
    case = s["case"]
    B, N, P, fmt, Hkv = case["B"], case["N"], case["P"], case["fmt"], case["Hkv"]
    every = torch.arange(256, device="cuda", dtype=torch.int32).to(torch.uint8).view(F8[fmt]).double()
    values = torch.unique(every[every.isfinite()])
    # halfway between two neighbours the one with the even code wins
    codes = values.to(F8[fmt]).view(torch.uint8)

    def nearest(x):
        hi = torch.searchsorted(values, x.contiguous()).clamp(1, len(values) - 1)
        a, b = values[hi - 1], values[hi]
        up = (b - x < x - a) | ((b - x == x - a) & (codes[hi] % 2 == 0))
        return torch.where(up, b, a)
    o = {}
    for pages, scale, tree in (("k_pages", "k_scale", "k_tree"), ("v_pages", "v_scale", "v_tree")):
        vals, sc = s[pages].double(), s[scale].double()
        for b in range(B):
            base, count = int(s["prefix_len"][b]), int(s["accept_len"][b]) + 1
            rows = s["path"][b, :count].long() if s["path"] is not None else torch.arange(count, device="cuda")
            for j in range(base // P, (base + count - 1) // P + 1):
                p = int(s["block_table"][b, j])
                lo, hi = max(base, j * P), min(base + count, j * P + P)
                x = s[tree][b, rows[lo - base:hi - base]].double().transpose(0, 1)  # [Hkv, rows, d]
                amax = x.abs().amax(dim=(1, 2))
                top = float(values[-1])
                k = torch.full((Hkv,), EXP_MIN, dtype=torch.float64, device="cuda")
                k = torch.where(amax > 0, torch.ceil(torch.log2(amax.clamp(min=1e-300) / top)), k).clamp(EXP_MIN, EXP_MAX)
                k = torch.where(amax > top * 2.0 ** k, k + 1, torch.where((amax > 0) & (amax <= top * 2.0 ** (k - 1)), k - 1, k))
                k = k.clamp(EXP_MIN, EXP_MAX)
                new = 2.0 ** k
                if lo > j * P:  # tokens already there: the scale never shrinks
                    grown = torch.maximum(sc[p], new)
                    old = vals[p, :, :lo - j * P]
                    vals[p, :, :lo - j * P] = torch.where((grown > sc[p])[:, None, None],
                                                          nearest(old.nan_to_num(0) * (sc[p] / grown)[:, None, None]), old)
                    new = grown
                vals[p, :, lo - j * P:hi - j * P] = nearest(x / new[:, None, None])
                sc[p] = new
        o[pages], o[scale] = vals, sc
    n = case["path_len"] or N
    o["new_prefix_len"] = s["prefix_len"].long() + s["accept_len"].long() + 1
    if s["feat_out"] is not None:
        feat = torch.zeros(B, n, case["F"], dtype=torch.float64, device="cuda")
        for b in range(B):
            count = int(s["accept_len"][b]) + 1
            feat[b, :count] = s["features"][b, s["path"][b, :count].long()].double()
        o["feat_out"] = feat
    return o
