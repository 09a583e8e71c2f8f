"""The paged 8-bit KV cache on the GPU against the CPU oracle: attention within
bounds derived from its roundings, the commit's codes and the block map
exactly."""
import numpy as np
import pytest
import torch

import oracle as O
from speculative_decoding_eagle_gb300 import binding as E
from tests.parity_util import ocfg

pytestmark = pytest.mark.gpu

F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731


def rounded(rng, dtype, *shape):
    """Normal values that the compute type holds exactly."""
    x = torch.from_numpy(rng.standard_normal(shape).astype(np.float32))
    return (x.bfloat16().float() if dtype == "bf16" else x).numpy()


def tdt(dtype):
    return torch.bfloat16 if dtype == "bf16" else torch.float32


class Pool:
    """Pages of random codes under scales from 2^-9 to 2^-5; what no sequence holds is stale: NaN codes too."""

    def __init__(self, rng, lens, P, Hkv, d, fmt, spare=3, exps=(-9, -5), interleave=True, cols=None):
        self.rng, self.lens, self.P, self.Hkv, self.d, self.fmt = rng, list(lens), P, Hkv, d, fmt
        blocks = [-(-max(n, 0) // P) for n in lens]
        self.cols = cols or max(1, max(blocks))
        self.pages = sum(blocks) + spare
        order = rng.permutation(self.pages)
        self.table = np.full((len(lens), self.cols), -1, np.int32)
        at = 0
        top = {"e4m3": 0x7E, "e5m2": 0x7B}[fmt]
        self.codes = [rng.integers(0, 256, (self.pages, Hkv, P, d)).astype(np.uint8) for _ in range(2)]
        self.scale = [(2.0 ** rng.integers(*exps, (self.pages, Hkv))).astype(np.float32) for _ in range(2)]
        self.room = 1.0 if fmt == "e4m3" else 2.0 ** -7
        for b, n in enumerate(blocks):
            self.table[b, :n] = order[at:at + n]
            at += n
            for j in range(n):
                p, fill = self.table[b, j], min(P, lens[b] - j * P)
                for c in self.codes:  # normal data, not raw codes
                    x = rng.standard_normal((Hkv, fill, d)) * 0.3 * O.paged_oracle.MAX_VALUE[fmt] * self.room
                    c[p, :, :fill] = O.encode(np.clip(x, -O.code_value(top, fmt), O.code_value(top, fmt)), fmt)
        self.free = list(order[at:])
        kv = torch.zeros(self.pages, 2, Hkv, P, d, dtype=torch.uint8, device="cuda")
        if not interleave:
            kv = torch.zeros(2, self.pages, Hkv, P, d, dtype=torch.uint8, device="cuda").transpose(0, 1)
        self.k, self.v = kv[:, 0].view(F8[fmt]), kv[:, 1].view(F8[fmt])
        self.ks, self.vs = dev(self.scale[0]), dev(self.scale[1])
        self.cache = E.PagedCache(self.k, self.v, self.ks, self.vs)
        self.upload()

    def upload(self):
        self.k.view(torch.uint8).copy_(torch.from_numpy(self.codes[0]))
        self.v.view(torch.uint8).copy_(torch.from_numpy(self.codes[1]))
        self.ks.copy_(torch.from_numpy(self.scale[0]))
        self.vs.copy_(torch.from_numpy(self.scale[1]))

    def host_codes(self):
        return [x.view(torch.uint8).cpu().numpy() for x in (self.k, self.v)]

    def sequence(self, b):
        n = max(self.lens[b], 0)
        return [O.dequantised(c, s, self.fmt, self.table[b], n) for c, s in zip(self.codes, self.scale)]


def random_tree(rng, B, N):
    keep = np.zeros((B, N, N), bool)
    for b in range(B):
        for i in range(N):
            if i:
                keep[b, i] = keep[b, rng.integers(max(0, i - 20), i)]
            keep[b, i, i] = True
    return keep


def mask_words(keep):
    B, N, _ = keep.shape
    W = (N + 63) // 64
    m = np.zeros((B, N, W), np.uint64)
    for w in range(W):
        for j in range(64 * w, min(N, 64 * w + 64)):
            m[:, :, w] |= keep[:, :, j].astype(np.uint64) << np.uint64(j - 64 * w)
    return m


def check_attention(got, glse, ref, d, dtype, L, rows):
    """|error| within what the roundings allow, element by element.

    A score is a sum of d products in fp32 and a few more roundings: (d + 8) 2^-24 of sum |q||k| * scale, and its
    image in 2^x of a few 2^-22 (the hardware base-2 exponential); both sums of weights run in fp32 over L + N terms
    of one sign each (2^-24 a term at the worst; the partial sums of a block tree lose less).  bf16: q meets cached codes
    in fp16, its row's largest element at 2^14 or above, so a bf16 value loses at most half of fp16's last step there,
    2^-25 / 2^14; or, with d = 128 and more than 16 rows per KV head, as two e4m3 terms, the largest above 224 and half
    a step of the second term 2^-10: 2^-10 / 224; weights that meet cached values are rounded to fp16 (2^-11), those that meet tree rows to bf16
    (2^-8), out to bf16 (2^-8)."""
    out, lse, abs_c, abs_t, reach, flat = ref
    eps = (d + 8) * 2.0 ** -24 * reach + 2.0 ** -19 + (0 if dtype != "bf16" else (2.0 ** -10 / 224 if d == 128 and rows > 16 else 2.0 ** -39) * flat)
    weight = (2 * eps).T[:, :, None] + min((L + 128) * 2.0 ** -24, 2.0 ** -16)
    if dtype == "bf16":
        tol = 2.0 ** -8 * np.abs(out) + (2.0 ** -11 + weight) * abs_c + (2.0 ** -8 + weight) * abs_t
    else:
        tol = 2.0 ** -23 * np.abs(out) + weight * (abs_c + abs_t)
    err = np.abs(got - out)
    worst = np.unravel_index(np.argmax(err - tol), err.shape)
    assert (err <= tol * 1.001 + 1e-30).all(), (worst, err[worst], tol[worst])
    empty = np.isneginf(lse)
    assert (np.isneginf(glse) == empty).all()
    lerr = np.abs(np.where(empty, 0, glse - np.where(empty, 0, lse)))
    ltol = eps + (L + 128) * 2.0 ** -24 + 2.0 ** -22 * np.abs(np.where(empty, 0, lse))
    assert (lerr <= ltol).all(), float((lerr - ltol).max())


def run_attention(pool, B, N, Hq, dtype, rng, keep, splits=0, mask=True, scale=None, max_prefix=None, q=None,
                  stream=None):
    Hkv, d = pool.Hkv, pool.d
    q = rounded(rng, dtype, B, N, Hq, d) if q is None else q
    kt, vt = rounded(rng, dtype, B, N, Hkv, d), rounded(rng, dtype, B, N, Hkv, d)
    shape = E.PagedAttnShape(B=B, N=N, Hq=Hq, max_blocks=pool.cols, dtype=E.ET_BF16 if dtype == "bf16" else E.ET_F32,
                             scale=scale or 0.0, max_prefix=max(0, max(pool.lens)) if max_prefix is None else max_prefix,
                             num_splits=splits)
    ws = E.new_workspace(E.et_tree_attention_paged_workspace_size(shape, pool.cache))
    out = torch.full((B, N, Hq, d), 7.0, dtype=tdt(dtype), device="cuda")
    lse = torch.full((B, Hq, N), 7.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (shape, pool.cache, dev(pool.table), dev(np.array(pool.lens, np.int32)), dev(q).to(tdt(dtype)),
            dev(kt).to(tdt(dtype)), dev(vt).to(tdt(dtype)),
            dev(mask_words(keep).view(np.int64)) if mask else None, out)
    E.et_tree_attention_paged(*args, lse=lse, ws=ws, dev_status=status, stream=stream)
    torch.cuda.synchronize()
    return dict(q=q, kt=kt, vt=vt, out=out, lse=lse, status=status, args=args, ws=ws, shape=shape)


def check_all(pool, r, keep, dtype, scale=None, sample_rows=None):
    got, glse = r["out"].double().cpu().numpy(), r["lse"].double().cpu().numpy()
    for b, L in enumerate(pool.lens):
        if L < 0:
            assert (got[b] == 7).all() and (glse[b] == 7).all()  # no sequence: left as it was
            continue
        kc, vc = pool.sequence(b)
        ref = O.paged_attention(r["q"][b], kc, vc, r["kt"][b], r["vt"][b], np.ones(L, bool), keep[b],
                                scale or pool.d ** -0.5)
        check_attention(got[b], glse[b], ref, pool.d, dtype, L, r["q"].shape[1] * r["q"].shape[2] // pool.Hkv)


ATTN_CASES = [  # lens, N, Hq, Hkv, d, P, dtype, fmt, splits
    ([0], 1, 4, 4, 128, 16, "bf16", "e4m3", 0),
    ([1], 1, 4, 4, 128, 16, "bf16", "e4m3", 0),
    ([0, 1, 15, 16, 17, 31, 32, 33, -1, 47, 48, 49, 63, 64, 65, 129], 1, 8, 2, 128, 16, "bf16", "e4m3", 0),
    ([257, 100, 0, 512], 1, 4, 4, 64, 48, "bf16", "e5m2", 0),
    ([700, 33], 1, 16, 1, 128, 64, "bf16", "e4m3", 3),
    ([301], 1, 28, 4, 128, 256, "bf16", "e4m3", 0),
    ([90, 200], 2, 28, 4, 128, 32, "bf16", "e5m2", 2),
    ([400], 17, 4, 4, 64, 16, "bf16", "e4m3", 0),
    ([0, 3, 700], 17, 4, 2, 128, 16, "bf16", "e4m3", 0),
    ([128, 129], 33, 2, 2, 128, 128, "bf16", "e4m3", 1),
    ([500, 64], 61, 2, 2, 128, 64, "bf16", "e4m3", 0),
    ([95, 512, -1], 61, 8, 2, 64, 48, "bf16", "e5m2", 4),
    ([321], 64, 4, 4, 128, 32, "bf16", "e4m3", 2),
    ([200], 81, 16, 2, 128, 128, "bf16", "e4m3", 0),
    ([77, 0], 128, 7, 1, 64, 80, "bf16", "e4m3", 0),
    ([40, 0, 129, -1], 17, 4, 4, 64, 16, "f32", "e5m2", 0),
    ([300, 65], 3, 8, 2, 128, 64, "f32", "e4m3", 0),
    ([33], 128, 4, 1, 64, 32, "f32", "e4m3", 0),
]


@pytest.mark.parametrize("lens,N,Hq,Hkv,d,P,dtype,fmt,splits", ATTN_CASES)
def test_attention_matches_oracle(lens, N, Hq, Hkv, d, P, dtype, fmt, splits):
    rng = np.random.default_rng(len(lens) * 1000 + N * 10 + d + P)
    pool = Pool(rng, lens, P, Hkv, d, fmt, interleave=N % 2 == 1)
    keep = random_tree(rng, len(lens), N)
    r = run_attention(pool, len(lens), N, Hq, dtype, rng, keep, splits)
    check_all(pool, r, keep, dtype)
    assert int(r["status"].item()) == 0
    again = [r["out"].clone(), r["lse"].clone()]
    E.et_tree_attention_paged(*r["args"], lse=r["lse"], ws=r["ws"], dev_status=r["status"])
    torch.cuda.synchronize()
    assert torch.equal(again[0], r["out"]) and torch.equal(again[1], r["lse"])  # the same bits, the workspace re-armed


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [1, 19, 70])
def test_attention_without_a_mask_is_a_chain(N, dtype):
    rng = np.random.default_rng(N)
    pool = Pool(rng, [50, 0], 16, 2, 128, "e4m3")
    keep = np.broadcast_to(np.tril(np.ones((N, N), bool)), (2, N, N))
    r = run_attention(pool, 2, N, 4, dtype, rng, keep, mask=False)
    check_all(pool, r, keep, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [1, 40])
def test_rows_without_a_key_are_zero(N, dtype):
    rng = np.random.default_rng(2)
    pool = Pool(rng, [0, 30], 16, 2, 64, "e4m3")
    keep = random_tree(rng, 2, N)
    keep[:, N // 2] = False
    keep[0, 0] = False
    r = run_attention(pool, 2, N, 4, dtype, rng, keep)
    check_all(pool, r, keep, dtype)
    assert (r["out"][0, N // 2] == 0).all() and torch.isneginf(r["lse"][0, :, N // 2]).all()


@pytest.mark.parametrize("N", [1, 30])
def test_scales_that_differ_by_many_powers(N):
    # V scales from 2^-40 to 2^38 and scores of several hundred: the weights must neither overflow nor vanish
    rng = np.random.default_rng(8)
    pool = Pool(rng, [200, 77], 16, 2, 128, "e4m3", exps=(-9, -5))
    pool.scale[1] = (2.0 ** rng.integers(-40, 39, pool.scale[1].shape)).astype(np.float32)
    pool.scale[0] *= 3.0  # K scales need not be powers of two
    pool.upload()
    keep = random_tree(rng, 2, N)
    r = run_attention(pool, 2, N, 4, "bf16", rng, keep, scale=0.5)
    check_all(pool, r, keep, "bf16", scale=0.5)


@pytest.mark.parametrize("mag", [2.0 ** -90, 2.0 ** 60])
def test_queries_of_any_magnitude(mag):
    rng = np.random.default_rng(9)
    pool = Pool(rng, [100], 32, 2, 128, "e4m3")
    pool.scale[0] = (pool.scale[0] / mag).astype(np.float32)
    pool.upload()
    keep = np.zeros((1, 5, 5), bool)  # cached tokens only: the tree's keys have no scale
    q = rounded(rng, "bf16", 1, 5, 4, 128) * np.float32(mag)
    r = run_attention(pool, 1, 5, 4, "bf16", rng, keep, q=q)
    check_all(pool, r, keep, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [1, 61])
def test_bad_pages_and_lengths_are_flagged_and_dropped(N, dtype):
    rng = np.random.default_rng(4)
    pool = Pool(rng, [100, 100, 100], 16, 2, 128, "e4m3")
    keep = random_tree(rng, 3, N)
    pool.table[0, 2], pool.table[1, 0] = -1, pool.pages  # tokens 32..47 and 0..15 are gone
    r = run_attention(pool, 3, N, 4, dtype, rng, keep, max_prefix=90)  # and every prefix is cut at 90
    assert int(r["status"].item()) == E.ET_DEV_BAD_INDEX
    got, glse = r["out"].double().cpu().numpy(), r["lse"].double().cpu().numpy()
    for b in range(3):
        there = np.arange(90)
        there = np.ones(90, bool) if b == 2 else (there // 16 != 2 if b == 0 else there // 16 != 0)
        pool.table[b] = np.where((pool.table[b] < 0) | (pool.table[b] >= pool.pages), 0, pool.table[b])
        kc, vc = [O.dequantised(c, s, pool.fmt, pool.table[b], 90) for c, s in zip(pool.codes, pool.scale)]
        vc, kc = np.where(there[None, :, None], vc, 0), np.where(there[None, :, None], kc, 0)
        ref = O.paged_attention(r["q"][b], kc, vc, r["kt"][b], r["vt"][b], there, keep[b], 128 ** -0.5)
        check_attention(got[b], glse[b], ref, 128, dtype, 90, 2 * N)


def test_nan_in_a_cached_value_reaches_its_rows_alone():
    rng = np.random.default_rng(6)
    pool = Pool(rng, [40, 40], 16, 2, 128, "e4m3")
    pool.codes[1][pool.table[0, 1], 1, 3, 5] = 0x7F  # V of token 19, head 1, dim 5 of sequence 0
    pool.upload()
    keep = random_tree(rng, 2, 20)
    r = run_attention(pool, 2, 20, 4, "bf16", rng, keep)
    nan = torch.isnan(r["out"])
    want = torch.zeros_like(nan)
    want[0, :, 2:4, 5] = True
    assert torch.equal(nan, want) and not torch.isnan(r["lse"]).any()


def test_nan_in_a_tree_row_reaches_its_descendants_alone():
    rng = np.random.default_rng(16)
    N = 40
    pool = Pool(rng, [40], 16, 2, 64, "e4m3")
    keep = random_tree(rng, 1, N)
    r = run_attention(pool, 1, N, 4, "bf16", rng, keep)
    clean = r["out"].clone()
    kt, vt = r["args"][5], r["args"][6]
    kt[0, 33, 0, 7] = float("nan")            # head 0 of the group pair: scores of row 33 and below it
    vt[0, 21, 1, 3] = float("inf")            # head 1, dim 3
    vt[0, 5, 1, 60] = float("nan")
    E.et_tree_attention_paged(*r["args"], lse=r["lse"], ws=r["ws"], dev_status=r["status"])
    torch.cuda.synchronize()
    want = clean.clone()
    sees = torch.from_numpy(keep[0]).cuda()
    want[0, sees[:, 33], 0:2] = float("nan")
    want[0, sees[:, 21], 2:4, 3] = float("inf")
    want[0, sees[:, 5], 2:4, 60] = float("nan")
    assert torch.equal(torch.isnan(want), torch.isnan(r["out"]))
    assert torch.equal(torch.nan_to_num(want, nan=0.0), torch.nan_to_num(r["out"], nan=0.0))


@pytest.mark.parametrize("N", [1, 61])
def test_pages_past_four_gigabytes(N):
    rng = np.random.default_rng(7)
    Hkv, P, d, L = 8, 64, 128, 200
    page = Hkv * P * d
    pages = (5 << 30) // page
    small = Pool(rng, [L], P, Hkv, d, "e4m3", spare=1)
    kv = torch.zeros(2, pages, Hkv, P, d, dtype=torch.uint8, device="cuda")
    scale = torch.ones(2, pages, Hkv, device="cuda")
    where = pages - 1 - np.arange(4, dtype=np.int32) * 7
    for j, p in enumerate(where):
        for x in range(2):
            kv[x, int(p)] = dev(small.codes[x][small.table[0, j]])
            scale[x, int(p)] = dev(small.scale[x][small.table[0, j]])
    far = Pool.__new__(Pool)
    far.__dict__.update(small.__dict__)
    far.cache = E.PagedCache(kv[0].view(F8["e4m3"]), kv[1].view(F8["e4m3"]), scale[0], scale[1])
    far.table = where[None]
    keep = random_tree(rng, 1, N)
    r = run_attention(far, 1, N, 8, "bf16", rng, keep)
    check_all(small, r, keep, "bf16")


def test_attention_on_another_stream_and_in_a_graph():
    rng = np.random.default_rng(11)
    pool = Pool(rng, [300, 90], 64, 2, 128, "e4m3")
    for N, splits in ((1, 2), (61, 2), (61, 1)):
        keep = random_tree(rng, 2, N)
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        r = run_attention(pool, 2, N, 4, "bf16", rng, keep, splits, stream=s)
        check_all(pool, r, keep, "bf16")
        want = [r["out"].clone(), r["lse"].clone()]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            E.et_tree_attention_paged(*r["args"], lse=r["lse"], ws=r["ws"], dev_status=r["status"])
        r["out"].zero_()
        for _ in range(3):
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(want[0], r["out"]) and torch.equal(want[1], r["lse"])


# ---------------------------------------------------------------------------
# commit
# ---------------------------------------------------------------------------
def run_commit(pool, tree, accept_len, path, prefix, dtype, features=None, feat=0):
    B, N = tree[0].shape[:2]
    path_len = 0 if path is None else path.shape[1]
    shape = E.PagedCommitShape(B=B, N=N, path_len=path_len, max_blocks=pool.cols,
                               dtype=E.ET_BF16 if dtype == "bf16" else E.ET_F32, feat_dim=feat)
    new = torch.full((B,), -77, dtype=torch.int32, device="cuda")
    fout = torch.full((B, path_len, feat), 5.0, dtype=tdt(dtype), device="cuda") if feat else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    E.et_kv_commit_paged(shape, pool.cache, dev(pool.table), dev(tree[0]).to(tdt(dtype)), dev(tree[1]).to(tdt(dtype)),
                         dev(np.asarray(accept_len, np.int32)), None if path is None else dev(path),
                         dev(np.asarray(prefix, np.int32)), new,
                         features=None if features is None else dev(features).to(tdt(dtype)), feat_out=fout,
                         dev_status=status)
    torch.cuda.synchronize()
    return new.cpu().numpy(), fout, int(status.item())


def check_codes(pool, tree, accept_len, path, prefix):
    codes = pool.host_codes()
    for x, (c, s) in enumerate(zip(codes, (pool.ks, pool.vs))):
        want_c, want_s = O.kv_commit_paged(pool.codes[x], pool.scale[x], pool.fmt, pool.table, tree[x],
                                           np.asarray(accept_len), path, np.asarray(prefix))
        # every byte of the pool: pages and rows that nobody appends to stay as they were
        nan = np.isnan(O.decode(want_c, pool.fmt))
        np.testing.assert_array_equal(np.isnan(O.decode(c, pool.fmt)), nan)
        np.testing.assert_array_equal(c[~nan], want_c[~nan])
        np.testing.assert_array_equal(s.cpu().numpy(), want_s)


def random_paths(rng, B, N, D, accept_len):
    path = np.full((B, D + 1), -1, np.int32)
    for b in range(B):
        if accept_len[b] >= 0:
            path[b, 0] = 0
            path[b, 1:accept_len[b] + 1] = np.sort(rng.choice(np.arange(1, N), accept_len[b], replace=False))
    return path


COMMIT_CASES = [  # B, N, Hkv, d, P, depth, dtype, fmt, F
    (1, 2, 1, 64, 16, 1, "bf16", "e4m3", 0),
    (9, 61, 4, 128, 16, 16, "bf16", "e4m3", 0),
    (9, 61, 4, 64, 16, 16, "f32", "e5m2", 64),
    (5, 61, 32, 128, 64, 6, "bf16", "e4m3", 4096),
    (5, 20, 2, 128, 48, 6, "f32", "e4m3", 0),
    (3, 17, 3, 64, 256, 4, "bf16", "e5m2", 8),
]


@pytest.mark.parametrize("B,N,Hkv,d,P,D,dtype,fmt,F", COMMIT_CASES)
def test_commit_matches_oracle(B, N, Hkv, d, P, D, dtype, fmt, F):
    rng = np.random.default_rng(B * 100 + N + P)
    alen = rng.integers(0, D + 1, B)
    alen[0] = D
    prefix = rng.integers(0, 3 * P, B)
    prefix[0] = P - 1                      # one row ends a page, the others begin the next
    if B > 4:
        prefix[1], prefix[2], prefix[3], alen[4] = 0, P, -1, -1
    pool = Pool(rng, list(prefix), P, Hkv, d, fmt, spare=3 * B, cols=6)
    for b in range(B):                     # room for the new rows
        for j in range(-(-max(prefix[b], 0) // P), -(-(max(prefix[b], 0) + D + 1) // P)):
            pool.table[b, j] = pool.free.pop()
    path = random_paths(rng, B, N, D, alen)
    # some heads outgrow their scale by much, some stay below it
    tree = [rounded(rng, dtype, B, N, Hkv, d) * (2.0 ** rng.integers(-12, 12, (B, 1, Hkv, 1))).astype(np.float32)
            for _ in range(2)]
    feats = rounded(rng, dtype, B, N, F) if F else None
    new, fout, status = run_commit(pool, tree, alen, path, prefix, dtype, feats, F)
    check_codes(pool, tree, alen, path, prefix)
    rows = np.where(prefix < 0, 0, alen + 1)
    np.testing.assert_array_equal(new, prefix + rows)
    assert status == 0
    if F:
        want = np.zeros((B, D + 1, F), np.float32)
        for b in range(B):
            want[b, :rows[b]] = feats[b, path[b, :rows[b]]]
        np.testing.assert_array_equal(fout.float().cpu().numpy(), want)


@pytest.mark.parametrize("P,dtype,fmt", [(16, "bf16", "e4m3"), (64, "f32", "e5m2"), (80, "bf16", "e4m3")])
def test_prompt_rows_in_order(P, dtype, fmt):
    rng = np.random.default_rng(P)
    B, N, Hkv, d = 4, 333, 2, 128
    alen, prefix = np.array([N - 1, -1, 100, 0]), np.array([5, 9, 0, P - 1])
    pool = Pool(rng, list(prefix), P, Hkv, d, fmt, spare=B * (N // P + 2), cols=N // P + 3)
    for b in range(B):
        for j in range(-(-prefix[b] // P), -(-(prefix[b] + N) // P)):
            pool.table[b, j] = pool.free.pop()
    tree = [rounded(rng, dtype, B, N, Hkv, d) for _ in range(2)]
    new, _, status = run_commit(pool, tree, alen, None, prefix, dtype)
    check_codes(pool, tree, alen, None, prefix)
    np.testing.assert_array_equal(new, prefix + alen + 1)
    assert status == 0


def test_commit_zero_huge_and_nonfinite_rows():
    rng = np.random.default_rng(12)
    B, N, Hkv, d, P = 4, 3, 1, 64, 16
    prefix, alen = np.array([0, 16, 3, 0]), np.array([1, 1, 1, 1])
    pool = Pool(rng, [0, 16, 3, 0], P, Hkv, d, "e4m3", spare=6, cols=2)
    for b, j in ((0, 0), (1, 1), (3, 0)):
        pool.table[b, j] = pool.free.pop()
    path = np.array([[0, 2]] * B, np.int32)
    tree = [rounded(rng, "bf16", B, N, Hkv, d) for _ in range(2)]
    for t in tree:
        t[0] = 0.0
        t[1, 0, 0, 3] = 2.0 ** 100  # past 448 * 2^48
        t[1, 2, 0, 4] = -2.0 ** 100
        t[2, 0, 0, 1], t[2, 2, 0, 2], t[2, 2, 0, 9] = np.nan, np.inf, -np.inf
        t[3] = np.nan
    _, _, status = run_commit(pool, tree, alen, path, prefix, "bf16")
    check_codes(pool, tree, alen, path, prefix)
    assert status == E.ET_DEV_NONFINITE
    assert pool.ks[pool.table[0, 0], 0].item() == 2.0 ** -48


def test_commit_onto_a_scale_of_another_origin():
    rng = np.random.default_rng(13)
    pool = Pool(rng, [20], 16, 2, 128, "e4m3", spare=1, cols=2)
    for s in pool.scale:
        s *= np.float32(1.7)
    pool.upload()
    tree = [rounded(rng, "f32", 1, 4, 2, 128) for _ in range(2)]
    path = np.array([[0, 1, 3]], np.int32)
    for t in tree:
        t *= 0.01  # below the scales that are there: they stay, and divide in fp32
    _, _, status = run_commit(pool, tree, [2], path, [20], "f32")
    check_codes(pool, tree, [2], path, [20])
    assert status == 0


def test_commit_skips_and_flags_bad_rows():
    rng = np.random.default_rng(14)
    B, N, P = 6, 5, 16
    prefix = np.array([3, 3, 3, 3, 40, 15])
    pool = Pool(rng, [3, 3, 3, 3, 16, 15], P, 2, 64, "e4m3", spare=2, cols=2)
    alen = np.array([1, 3, -2, 1, 0, 1])           # path_len 3: 3 and -2 are no lengths
    path = np.array([[0, 9, -1], [0, 1, 2], [0, 1, 2], [0, 2, -1], [0, -1, -1], [0, 1, -1]], np.int32)
    pool.table[3, 0] = pool.pages                  # no page of the cache
    pool.table[5, 1] = -1                          # position 15 fits, 16 has no page; sequence 4 is past its table
    tree = [rounded(rng, "bf16", B, N, 2, 64) for _ in range(2)]
    before = pool.host_codes()
    new, _, status = run_commit(pool, tree, alen, path, prefix, "bf16")
    assert status == E.ET_DEV_BAD_INDEX
    np.testing.assert_array_equal(new, [5, -77, -77, 5, 41, 17])
    ok_alen, ok_prefix = np.array([0, -1, -1, -1, -1, 0]), np.array([3, 3, 3, 3, 16, 15])
    check_codes(pool, tree, ok_alen, path, ok_prefix)  # row 9, sequences 1 to 4 and position 16 were skipped
    assert before[0].shape == pool.host_codes()[0].shape


# ---------------------------------------------------------------------------
# block map
# ---------------------------------------------------------------------------
class Map:
    def __init__(self, B, cols, pool, max_new, P):
        i32 = dict(dtype=torch.int32, device="cuda")
        self.shape = E.BlockMapShape(B=B, page_size=P, max_blocks=cols, num_pages=pool, max_new=max_new)
        self.n, self.table = torch.zeros(B, **i32), torch.full((B, cols), -1, **i32)
        self.free, self.count = torch.arange(pool, **i32), torch.full((1,), pool, **i32)
        self.slots = torch.full((B, max_new), -5, dtype=torch.int64, device="cuda") if max_new else None
        self.status = torch.zeros(1, **i32)

    def step(self, lens, new):
        self.status.zero_()
        n, table = self.n.cpu().numpy(), self.table.cpu().numpy()
        free = self.free.cpu().numpy()[:int(self.count)].tolist()
        stale = self.free.cpu().numpy()
        E.et_block_map(self.shape, dev(np.asarray(lens, np.int32)), dev(np.asarray(new, np.int32)), self.n, self.table,
                       self.free, self.count, self.slots, dev_status=self.status)
        torch.cuda.synchronize()
        n, table, left, slots, short, bad = O.block_map(lens, new, n, table, free, self.shape.page_size,
                                                        self.shape.max_new)
        np.testing.assert_array_equal(self.n.cpu().numpy(), n)
        np.testing.assert_array_equal(self.table.cpu().numpy(), table)
        assert int(self.count) == len(left)
        got = self.free.cpu().numpy()
        np.testing.assert_array_equal(got[:len(left)], left)
        np.testing.assert_array_equal(got[len(left):], stale[len(left):])
        if self.slots is not None:
            np.testing.assert_array_equal(self.slots.cpu().numpy(), slots)
        assert int(self.status.item()) == (E.ET_DEV_NO_PAGES if short else 0) | (E.ET_DEV_BAD_INDEX if bad else 0)
        return short


@pytest.mark.parametrize("B,P,L,max_new,share", [(1, 16, 40, 1, 1.0), (7, 64, 900, 61, 1.0), (33, 48, 500, 128, 0.4),
                                                 (33, 16, 300, 0, 0.3), (1030, 16, 200, 5, 0.6), (4096, 32, 70, 3, 0.5),
                                                 (2, 1, 3000, 3000, 0.7)])
def test_block_map_matches_oracle_over_many_steps(B, P, L, max_new, share):
    rng = np.random.default_rng(B + P)
    cols = -(-(L + max(max_new, 4)) // P)
    m = Map(B, cols, max(1, int(share * B * cols)), max_new, P)
    lens = rng.integers(0, L + 1, B)
    shorts = 0
    for step in range(6):
        shorts += m.step(lens, rng.integers(0, max(max_new, 4) + 1, B))
        u = rng.random(B)
        lens = np.where(u < 0.6, np.minimum(lens + rng.integers(0, 9, B), L), lens)
        lens = np.where(u > 0.9, rng.integers(0, L + 1, B), lens)
        lens = np.where((u > 0.6) & (u < 0.75), 0, lens)
        lens = np.where((u > 0.75) & (u < 0.8), -1, lens)
        lens = np.where((u > 0.8) & (lens < 0), 1, lens)
    m.step(np.zeros(B, int), np.zeros(B, int))  # everyone ends: all pages are back, each once
    assert share < 1 or shorts == 0
    assert sorted(m.free.cpu().numpy()[:int(m.count)].tolist()) == list(range(m.shape.num_pages))


def test_block_map_flags_bad_arguments():
    m = Map(5, 4, 30, 6, 16)
    m.step([10, 60, 3, 20, 0], [1, 4, 0, 6, 0])
    m.n[2] = 9  # more blocks than the table has columns
    m.step([10, 60, 3, 20, 0], [1, 5, 1, 7, -1])  # 65 tokens do not fit four pages; 7 and -1 are no counts
    assert int(m.status.item()) == E.ET_DEV_BAD_INDEX
    m.count.fill_(99)  # more free pages than there are: clamped
    m.status.zero_()
    before = m.table.clone()
    E.et_block_map(m.shape, dev(np.full(5, -1, np.int32)), dev(np.zeros(5, np.int32)), m.n, m.table, m.free, m.count,
                   m.slots, dev_status=m.status)
    assert int(m.status.item()) == E.ET_DEV_BAD_INDEX and int(m.count) == 30 and torch.equal(before, m.table)


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
def test_a_served_batch_over_several_steps():
    """Prompts, then verification steps: pages mapped, attention over them, greedy acceptance, commit; one request
    ends on the way and another takes its pages.  The cache is followed by the oracle bit for bit."""
    rng = np.random.default_rng(21)
    B, N, Hq, Hkv, d, P, V, D = 3, 9, 4, 2, 128, 16, 200, 3
    cols, pages = 8, 20
    m = Map(B, cols, pages, 64, P)
    cache = E.PagedCache.allocate(pages, Hkv, P, d)
    codes = [np.zeros((pages, Hkv, P, d), np.uint8) for _ in range(2)]
    scale = [np.ones((pages, Hkv), np.float32) for _ in range(2)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def commit(N, lens, alen, path, dlens, dalen, dpath):
        tree = [rounded(rng, "bf16", B, N, Hkv, d) * np.float32(2.0 ** rng.integers(-2, 3)) for _ in range(2)]
        shape = E.PagedCommitShape(B=B, N=N, path_len=0 if path is None else D + 1, max_blocks=cols)
        new = torch.zeros(B, dtype=torch.int32, device="cuda")
        E.et_kv_commit_paged(shape, cache, m.table, dev(tree[0]).bfloat16(), dev(tree[1]).bfloat16(), dalen, dpath, dlens,
                             new, dev_status=status)
        torch.cuda.synchronize()
        table = m.table.cpu().numpy()
        for x in range(2):
            codes[x], scale[x] = O.kv_commit_paged(codes[x], scale[x], "e4m3", table, tree[x], alen, path, lens)
        for x, (c, s) in enumerate(((cache.k_pages, cache.k_scale), (cache.v_pages, cache.v_scale))):
            np.testing.assert_array_equal(c.view(torch.uint8).cpu().numpy(), codes[x])
            np.testing.assert_array_equal(s.cpu().numpy(), scale[x])
        return new

    lens = np.zeros(B, np.int64)
    prompt = np.array([37, 5, 50])
    assert not m.step(lens, prompt)
    dlens = commit(50, lens, prompt - 1, None, dev(lens.astype(np.int32)), dev((prompt - 1).astype(np.int32)), None)
    lens = lens + prompt
    np.testing.assert_array_equal(dlens.cpu().numpy(), lens)
    cfg = E.TreeCfg(B=B, V=V, depth=D, topk=2, m=2, n=N - 1)
    parent = np.array([-1, 0, 0, 1, 1, 2, 3, 3, 5], np.int32)
    rank = np.array([-1, 0, 1, 0, 1, 0, 0, 1, 0], np.int32)
    ws_tree = E.new_workspace(E.et_tree_workspace_size(cfg))
    for step in range(4):
        if step == 2:  # request 1 ends, and its place is taken by a prompt of 30
            lens[1] = 0
            assert not m.step(lens, np.array([0, 0, 0]))
            assert not m.step(lens, np.array([0, 30, 0]))
            alen = np.array([-1, 29, -1])
            dlens = commit(30, lens, alen, None, dev(lens.astype(np.int32)), dev(alen.astype(np.int32)), None)
            lens = lens + alen + 1
        assert not m.step(lens, np.full(B, D + 1))
        # the tree, its mask and the attention over the paged prefix
        draft = (rng.standard_normal((B * N, V)) * 3).astype(np.float32)
        rmap = np.arange(B * N, dtype=np.int32).reshape(B, N)
        tb = E.TreeBuffers.allocate_flat(B, N, root_tok=dev(np.arange(B, dtype=np.int32)))
        E.et_static_tree(B, V, 2, dev(parent), dev(rank), dev(draft), dev(rmap), tb, dev_status=status)
        mask = torch.zeros((B, N, 1), dtype=torch.int64, device="cuda")
        pos = torch.zeros((B, N), dtype=torch.int32, device="cuda")
        E.et_tree_mask_posids(cfg, tb, dlens, mask, pos)
        q, kt, vt = (rounded(rng, "bf16", B, N, h, d) for h in (Hq, Hkv, Hkv))
        shape = E.PagedAttnShape(B=B, N=N, Hq=Hq, max_blocks=cols, max_prefix=cols * P)
        ws = E.new_workspace(E.et_tree_attention_paged_workspace_size(shape, cache))
        out = torch.zeros((B, N, Hq, d), dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros((B, Hq, N), device="cuda")
        E.et_tree_attention_paged(shape, cache, m.table, dlens, dev(q).bfloat16(), dev(kt).bfloat16(),
                                  dev(vt).bfloat16(), mask, out, lse=lse, ws=ws, dev_status=status)
        bits = mask.cpu().numpy().view(np.uint64)[:, :, 0]
        keep = ((bits[:, :, None] >> np.arange(N, dtype=np.uint64)) & np.uint64(1)).astype(bool)
        table = m.table.cpu().numpy()
        for b in range(B):
            kc, vc = [O.dequantised(c, s, "e4m3", table[b], int(lens[b])) for c, s in zip(codes, scale)]
            ref = O.paged_attention(q[b], kc, vc, kt[b], vt[b], np.ones(lens[b], bool), keep[b], d ** -0.5)
            check_attention(out[b].double().cpu().numpy(), lse[b].double().cpu().numpy(), ref, d, "bf16", int(lens[b]),
                            N * Hq // Hkv)
        # greedy acceptance against a target that mostly agrees, then the commit of its path
        target = (draft + 0.2 * rng.standard_normal(draft.shape)).astype(np.float32)
        alen = torch.zeros(B, dtype=torch.int32, device="cuda")
        path = torch.zeros((B, D + 1), dtype=torch.int32, device="cuda")
        toks = torch.zeros((B, D + 1), dtype=torch.int32, device="cuda")
        E.et_verify_accept(cfg, E.ET_ACCEPT_GREEDY, tb, dev(target), alen, path, toks, ws_tree)
        halen, hpath = alen.cpu().numpy(), path.cpu().numpy()
        assert ocfg(cfg).n == N - 1 and halen.max() > 0
        dlens = commit(N, lens, halen, hpath, dlens, alen, path)
        lens = lens + halen + 1
        np.testing.assert_array_equal(dlens.cpu().numpy(), lens)
    assert int(status.item()) == 0


# ---------------------------------------------------------------------------
# many sequences, many chunks, shared workspaces, waits that run out
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("B,N,Hq,Hkv,d", [(150, 1, 2, 1, 128), (150, 9, 4, 2, 64), (650, 17, 1, 1, 128)])
def test_batches_past_one_block_of_lengths(B, N, Hq, Hkv, d):
    # the kernels read a batch's lengths with one thread each up to their block's size, else take the bound
    rng = np.random.default_rng(B + N)
    lens = rng.integers(-1, 60, B)
    lens[B // 2], lens[-1] = 300, 200
    pool = Pool(rng, list(lens), 16, Hkv, d, "e4m3")
    keep = random_tree(rng, B, N)
    r = run_attention(pool, B, N, Hq, "bf16", rng, keep, splits=3)
    picked = [0, 1, B // 2, B // 2 + 1, B - 2, B - 1]
    got, glse = r["out"].double().cpu().numpy(), r["lse"].double().cpu().numpy()
    for b in picked:
        if lens[b] < 0:
            assert (got[b] == 7).all()
            continue
        kc, vc = pool.sequence(b)
        ref = O.paged_attention(r["q"][b], kc, vc, r["kt"][b], r["vt"][b], np.ones(lens[b], bool), keep[b], d ** -0.5)
        check_attention(got[b], glse[b], ref, d, "bf16", int(lens[b]), N * Hq // Hkv)
    assert int(r["status"].item()) == 0


@pytest.mark.parametrize("splits,chunks", [(3, 3), (8, 8), (9, 9), (13, 13), (40, 14)])
def test_chunks_that_form_a_cluster_and_more_that_use_the_workspace(splits, chunks):
    """Up to eight chunks merge through shared memory, more through the workspace; some have no keys, some half a tile."""
    rng = np.random.default_rng(29)
    lens = [1700, 0, 1, 300, 1664]
    pool = Pool(rng, lens, 48, 2, 128, "e4m3")
    keep = random_tree(rng, 5, 37)
    runs = [run_attention(pool, 5, 37, 4, "bf16", rng, keep, splits) for _ in range(2)]
    assert E.et_tree_attention_paged_splits(runs[0]["shape"], pool.cache) == chunks
    graphs = []
    for r in runs:
        check_all(pool, r, keep, "bf16")
        r["want"] = r["out"].clone()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):  # both on one workspace
            E.et_tree_attention_paged(*r["args"], lse=r["lse"], ws=runs[0]["ws"], dev_status=r["status"])
    for r in runs:
        r["out"].zero_()
    for _ in range(4):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for r in runs:
        assert torch.equal(r["out"], r["want"]) and int(r["status"].item()) == 0


@pytest.mark.parametrize("N,Hq,Hkv,d", [(1, 4, 2, 128), (5, 6, 2, 128), (30, 2, 1, 128), (1, 2, 2, 64), (30, 2, 1, 64),
                                        (70, 1, 1, 64)])
@pytest.mark.parametrize("splits", [2, 3, 5, 8])
def test_one_sequence_whose_chunks_merge_as_a_cluster(N, Hq, Hkv, d, splits):
    """One graph, the prefix it was captured with and shorter ones, which leave blocks of the cluster without keys."""
    rng = np.random.default_rng(47)
    pool = Pool(rng, [1100], 48, Hkv, d, "e4m3")
    keep = random_tree(rng, 1, N)
    r = run_attention(pool, 1, N, Hq, "bf16", rng, keep, splits)
    assert E.et_tree_attention_paged_splits(r["shape"], pool.cache) == splits
    assert E.et_tree_attention_paged_workspace_size(r["shape"], pool.cache) == 0
    check_all(pool, r, keep, "bf16")
    want = r["out"].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        E.et_tree_attention_paged(*r["args"], lse=r["lse"], ws=r["ws"], dev_status=r["status"])
    for L in (0, 1, 31, 128, 140, 700, -1, 1100):
        r["args"][3].fill_(L)
        r["out"].fill_(7.0)
        r["lse"].fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        pool.lens = [L]
        check_all(pool, r, keep, "bf16")
    assert torch.equal(r["out"], want) and int(r["status"].item()) == 0


def test_one_workspace_serves_calls_of_different_shapes():
    """What one call leaves in a workspace of the largest size is no other call's counter."""
    rng = np.random.default_rng(43)
    pool = Pool(rng, [2100, 700], 48, 4, 128, "e4m3")
    small = Pool(rng, [900] + [40] * 30, 16, 4, 128, "e4m3")
    runs = []
    for p, N, splits in ((pool, 1, 5), (small, 1, 2), (pool, 61, 12), (pool, 2, 0), (small, 4, 7)):
        keep = random_tree(rng, len(p.lens), N)
        r = run_attention(p, len(p.lens), N, 4, "bf16", rng, keep, splits)
        check_all(p, r, keep, "bf16")
        runs.append(dict(r, want=r["out"].clone()))
    ws = E.new_workspace(max(r["ws"].numel() for r in runs))
    for r in runs + runs[::-1]:
        r["out"].zero_()
        E.et_tree_attention_paged(*r["args"], lse=r["lse"], ws=ws, dev_status=r["status"])
        torch.cuda.synchronize()
        assert torch.equal(r["out"], r["want"]) and int(r["status"].item()) == 0


SHARED = [  # lens: sequences whose lengths decide how many blocks each has
    [2100, -1, 0, 1, 700, 64, 2048],
    [2048, 2048],
    [-1, 2500, -1],
    [5000, 33, 32, 31],
    [int(n) for n in np.random.default_rng(1).integers(0, 900, 31)] + [2049],
]


@pytest.mark.parametrize("lens", SHARED, ids=lambda v: f"{len(v)}x{max(v)}")
@pytest.mark.parametrize("N,Hq,Hkv,d,fmt", [(1, 4, 2, 128, "e4m3"), (1, 2, 1, 64, "e5m2"), (20, 1, 1, 64, "e4m3"),
                                            (60, 1, 1, 64, "e4m3")])
def test_a_batch_shared_out_by_its_lengths(lens, N, Hq, Hkv, d, fmt):
    """One graph serves the lengths it was captured with and others; the share is worked out on the device."""
    rng = np.random.default_rng(41)
    B = len(lens)
    pool = Pool(rng, lens, 48, Hkv, d, fmt)
    keep = random_tree(rng, B, N)
    r = run_attention(pool, B, N, Hq, "bf16", rng, keep)
    assert E.et_tree_attention_paged_splits(r["shape"], pool.cache) > 1
    check_all(pool, r, keep, "bf16")
    want = r["out"].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        E.et_tree_attention_paged(*r["args"], lse=r["lse"], ws=r["ws"], dev_status=r["status"])
    prefix, first = r["args"][3], list(lens)
    for other in ([n // 3 if n > 0 else n for n in lens], [min(n, 0) for n in lens], [-1] * B, first):
        prefix.copy_(torch.tensor(other, dtype=torch.int32))
        r["out"].fill_(7.0)
        r["lse"].fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        pool.lens = other
        check_all(pool, r, keep, "bf16")
    assert torch.equal(r["out"], want) and int(r["status"].item()) == 0


@pytest.mark.parametrize("N,Hq,Hkv,d", [(1, 4, 2, 128), (30, 2, 1, 128), (30, 2, 1, 64), (70, 1, 1, 64)])
@pytest.mark.parametrize("splits", [1, 2, 7, 64, 1000])
def test_every_number_of_chunks_gives_the_same_sums(N, Hq, Hkv, d, splits):
    rng = np.random.default_rng(3)
    pool = Pool(rng, [900, 1, 130], 48, Hkv, d, "e5m2")
    keep = random_tree(rng, 3, N)
    r = run_attention(pool, 3, N, Hq, "bf16", rng, keep, splits)
    assert E.et_tree_attention_paged_splits(r["shape"], pool.cache) <= 64
    check_all(pool, r, keep, "bf16")


@pytest.mark.parametrize("N", [1, 61])
def test_a_loose_prefix_bound_changes_nothing_but_the_plan(N):
    rng = np.random.default_rng(5)
    pool = Pool(rng, [100, 40], 16, 2, 128, "e4m3", cols=400)
    keep = random_tree(rng, 2, N)
    r = run_attention(pool, 2, N, 4, "bf16", rng, keep, max_prefix=6000)
    check_all(pool, r, keep, "bf16")
    assert int(r["status"].item()) == 0


@pytest.mark.parametrize("N", [1, 61])
def test_graphs_and_streams(N):
    """Two captured graphs that use one workspace one after the other, and two streams with one each."""
    rng = np.random.default_rng(23)
    pool = Pool(rng, [500, 90], 32, 2, 128, "e4m3")
    keep = random_tree(rng, 2, N)
    runs = [run_attention(pool, 2, N, 4, "bf16", rng, keep, splits=3) for _ in range(2)]
    want = [r["out"].clone() for r in runs]
    graphs = []
    for r in runs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            E.et_tree_attention_paged(*r["args"], lse=r["lse"], ws=runs[0]["ws"], dev_status=r["status"])
        graphs.append(g)
    for _ in range(5):
        for r, g in zip(runs, graphs):
            r["out"].zero_()
            g.replay()
    torch.cuda.synchronize()
    for r, w in zip(runs, want):
        assert torch.equal(r["out"], w)
        r["out"].zero_()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for r, s in zip(runs, streams):
            E.et_tree_attention_paged(*r["args"], lse=r["lse"], ws=r["ws"], dev_status=r["status"], stream=s)
    torch.cuda.synchronize()
    for r, w in zip(runs, want):
        assert torch.equal(r["out"], w) and int(r["status"].item()) == 0


@pytest.mark.parametrize("N,d,splits", [(1, 128, 1), (1, 128, 3), (61, 128, 1), (61, 128, 3), (61, 64, 2)])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(N, d, splits):
    rng = np.random.default_rng(17)
    pool = Pool(rng, [900, 300], 64, 2, d, "e4m3")
    keep = random_tree(rng, 2, N)
    r = run_attention(pool, 2, N, 4, "bf16", rng, keep, splits)
    want = r["out"].clone()
    before = E.et_set_wait_limit(1)
    try:
        for _ in range(3):
            E.et_tree_attention_paged(*r["args"], lse=r["lse"], ws=r["ws"], dev_status=r["status"])
        torch.cuda.synchronize()
    finally:
        E.et_set_wait_limit(before if before < 1 << 32 else 0)
    # one wait may last some microseconds by itself: the mma.sync kernel's copies may land within its first
    status = int(r["status"].item())
    assert status == E.ET_DEV_TIMEOUT or (status == 0 and (N == 1 or d == 64) and torch.equal(r["out"], want))
    r["status"].zero_()
    E.et_tree_attention_paged(*r["args"], lse=r["lse"], ws=r["ws"], dev_status=r["status"])
    torch.cuda.synchronize()
    assert torch.equal(r["out"], want) and int(r["status"].item()) == 0


def test_commit_and_map_in_a_graph():
    """A captured step that maps a block, commits a path and maps again replays like eager calls."""
    rng = np.random.default_rng(31)
    B, N, Hkv, d, P, D, cols = 3, 9, 2, 64, 16, 3, 4
    m = Map(B, cols, B * cols, D + 1, P)
    cache = E.PagedCache.allocate(B * cols, Hkv, P, d, torch.float8_e5m2)
    lens = torch.tensor([14, 0, 15], dtype=torch.int32, device="cuda")
    new, more = torch.full_like(lens, D + 1), torch.zeros_like(lens)
    kt, vt = (dev(rounded(rng, "bf16", B, N, Hkv, d)).bfloat16() for _ in range(2))
    path = torch.tensor([[0, 2, 5, 7]] * B, dtype=torch.int32, device="cuda")
    alen = torch.tensor([3, 1, 2], dtype=torch.int32, device="cuda")
    shape = E.PagedCommitShape(B=B, N=N, path_len=D + 1, max_blocks=cols)

    def step():
        E.et_block_map(m.shape, lens, new, m.n, m.table, m.free, m.count, m.slots, dev_status=m.status)
        E.et_kv_commit_paged(shape, cache, m.table, kt, vt, alen, path, lens, more, dev_status=m.status)
        lens.copy_(more)
    first = [t.clone() for t in (lens, m.n, m.table, m.free, m.count)]
    for _ in range(3):
        step()
    torch.cuda.synchronize()
    want = [t.clone() for t in (lens, m.n, m.table, m.free, m.count, m.slots, cache.k_pages.view(torch.uint8),
                                cache.v_pages.view(torch.uint8), cache.k_scale, cache.v_scale)]
    for t, f in zip((lens, m.n, m.table, m.free, m.count), first):
        t.copy_(f)
    cache.k_pages.view(torch.uint8).zero_()
    cache.v_pages.view(torch.uint8).zero_()
    cache.k_scale.fill_(1)
    cache.v_scale.fill_(1)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    got = (lens, m.n, m.table, m.free, m.count, m.slots, cache.k_pages.view(torch.uint8),
           cache.v_pages.view(torch.uint8), cache.k_scale, cache.v_scale)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert int(m.status.item()) == 0
