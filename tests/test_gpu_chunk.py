"""Chunk attention over the paged 8-bit cache on the GPU, against the formula in 64 bits.

Tolerances: cached values are exact (codes times powers of two).  fp32: products and sums of up to 10^3 terms of order
one, each with a relative error of 2^-24, and exponentials of two with 2^-22: 2e-5 of the row's largest value leaves
room.  bf16: the weights are rounded to 8 bits (bf16) or 11 (fp16) and the result to 8 bits; a rounding is off by 2^-9 of
the value at most (half a step), so |out - exact| <= 2^-9 |exact| + 2^-9 sum_j p_j |v_j|: the second term is computed
beside the output and both are taken twice.
"""
import math

import pytest
import torch

from speculative_decoding_eagle_gb300 import binding as E

pytestmark = pytest.mark.gpu
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
DT = {"bf16": (E.ET_BF16, torch.bfloat16), "f32": (E.ET_F32, torch.float32)}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_eagle_gb300 import build_lib
    build_lib.build()
    E.load()


class Batch:
    """A batch's cache, rows and outputs; ``prefix`` < 0 marks an absent sequence, spare rows stand behind the last."""

    def __init__(self, prefix, rows, Hq, Hkv, d, P, fmt="e4m3", dtype="bf16", seed=0, spare=3, scale_exp=(-9, -4), stale="any"):
        g = torch.Generator(device="cuda")
        g.manual_seed(1000 + seed)
        self.prefix, self.rows, self.Hq, self.Hkv, self.d, self.P, self.fmt = prefix, rows, Hq, Hkv, d, P, fmt
        self.dt, dt = DT[dtype]
        B = len(prefix)
        blocks = [max(0, -(-n // P)) for n in prefix]
        cols = max(1, max(blocks))
        pages = sum(blocks) + 2
        order = torch.randperm(pages, generator=g, device="cuda")
        table = torch.full((B, cols), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(blocks):
            table[b, :n] = order[at:at + n].to(torch.int32)
            at += n
        self.table = table
        codes = lambda: torch.randint(0, 256, (pages, Hkv, P, d), generator=g, device="cuda", dtype=torch.int32).to(torch.uint8)  # noqa: E731
        self.cache = E.PagedCache.allocate(pages, Hkv, P, d, F8[fmt])
        top = {"e4m3": 448.0, "e5m2": 57344.0}[fmt]
        for pg, sc in ((self.cache.k_pages, self.cache.k_scale), (self.cache.v_pages, self.cache.v_scale)):
            x = (torch.randn(pages, Hkv, P, d, generator=g, device="cuda") * (top / 5)).clamp(-top, top)
            pg.view(torch.uint8).copy_(x.to(F8[fmt]).view(torch.uint8))
            lo, hi = scale_exp if fmt == "e4m3" else (scale_exp[0] - 7, scale_exp[1] - 7)
            sc.copy_(2.0 ** torch.randint(lo, hi + 1, sc.shape, generator=g, device="cuda").float())
        stale_codes = codes()  # NaN codes too
        for b, n in enumerate(prefix):
            if n > 0 and n % P:
                for pg in (self.cache.k_pages, self.cache.v_pages):
                    pg.view(torch.uint8)[table[b, n // P].long(), :, n % P:] = stale_codes[0, :, n % P:]
        T = sum(rows) + spare
        self.T = T
        start = [0]
        for r in rows:
            start.append(start[-1] + r)
        self.start = torch.tensor(start, dtype=torch.int32, device="cuda")
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dt)  # noqa: E731
        qkv = rnd(T, Hq + 2 * Hkv, d)
        self.q, self.k, self.v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        self.plen = torch.tensor(prefix, dtype=torch.int32, device="cuda")
        self.out = torch.full((T, Hq, d), 7.0, dtype=dt, device="cuda")
        self.lse = torch.full((T, Hq), 7.0, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self, splits=0, max_prefix=None, max_rows=None, ws=None, stream=None, scale=0.0):
        shape = E.ChunkAttnShape(B=len(self.prefix), rows=self.T, Hq=self.Hq, max_rows=max_rows or max(1, max(self.rows)),
                                 max_blocks=self.table.shape[1], dtype=self.dt, num_splits=splits, max_prefix=max_prefix,
                                 scale=scale)
        if ws is None:
            ws = E.new_workspace(E.et_chunk_attention_paged_workspace_size(shape, self.cache))
        E.et_chunk_attention_paged(shape, self.cache, self.table, self.plen, self.start, self.q, self.k, self.v, self.out,
                                   lse=self.lse, ws=ws, dev_status=self.status, stream=stream)
        torch.cuda.synchronize()
        return ws

    def exact(self, scale=None):
        """Per row: the output, the log-sum-exp, and sum_j p_j |v_j| (absent rows keep 7)."""
        out = torch.full(self.out.shape, 7.0, dtype=torch.float64, device="cuda")
        lse = torch.full(self.lse.shape, 7.0, dtype=torch.float64, device="cuda")
        mass = torch.zeros_like(out)
        G = self.Hq // self.Hkv
        scale = scale or 1 / math.sqrt(self.d)
        for b, n in enumerate(self.prefix):
            r0, r1 = int(self.start[b]), int(self.start[b + 1])
            if n < 0 or r1 == r0:
                continue
            pages = self.table[b, :-(-n // self.P)].long()
            sees = torch.cat([torch.ones(r1 - r0, n, dtype=torch.bool, device="cuda"),
                              torch.ones(r1 - r0, r1 - r0, dtype=torch.bool, device="cuda").tril()], 1)
            for g in range(self.Hkv):
                def column(codes, sc, new):
                    x = codes.view(torch.uint8)[pages, g].view(codes.dtype).double() * sc[pages, g].double()[:, None, None]
                    return torch.cat([x.reshape(-1, self.d)[:n], new[r0:r1, g].double()])
                k = column(self.cache.k_pages, self.cache.k_scale, self.k)
                v = column(self.cache.v_pages, self.cache.v_scale, self.v)
                z = torch.einsum("nhd,td->hnt", self.q[r0:r1, g * G:(g + 1) * G].double(), k) * scale
                z = torch.where(sees[None], z, -math.inf)
                total = torch.logsumexp(z, -1)
                p = torch.where(sees[None], torch.exp(z - total[..., None]), 0.0)
                out[r0:r1, g * G:(g + 1) * G] = torch.einsum("hnt,td->nhd", p, v)
                mass[r0:r1, g * G:(g + 1) * G] = torch.einsum("hnt,td->nhd", p, v.abs())
                lse[r0:r1, g * G:(g + 1) * G] = total.T
        return out, lse, mass

    def check(self, scale=None, status=0):
        out, lse, mass = self.exact(scale)
        assert int(self.status.item()) == status
        err = (self.out.double() - out).abs()
        if self.dt == E.ET_F32:
            assert bool((err <= 2e-5 * out.abs().amax(-1, keepdim=True)).all()), float(err.max())
        else:
            over = err - 2 * 2.0 ** -9 * (out.abs() + mass)
            assert bool((over <= 0).all()), (float(over.max()), float(err.max()))
        assert bool(((self.lse.double() - lse).abs() <= 1e-5 * (1 + lse.abs())).all()), float((self.lse.double() - lse).abs().max())


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("prefix,rows,Hq,Hkv,P", [
    ([0], [1], 4, 4, 16),                                   # one token, nothing before it
    ([1], [1], 4, 2, 16),
    ([37], [1], 8, 1, 32),
    ([128], [128], 2, 2, 64),                               # whole tiles
    ([127], [129], 2, 2, 64),
    ([129], [127], 4, 4, 48),                               # pages that do not divide a tile
    ([300], [257], 4, 2, 16),
    ([0], [513], 3, 3, 64),
    ([1000], [65], 14, 2, 128),                             # seven heads to a KV head
    ([640], [31], 16, 1, 64),                               # sixteen
    ([5, 0, -1, 260, 90], [1, 200, 40, 0, 3], 4, 2, 32),    # absent and idle sequences
])
def test_matches_the_formula(prefix, rows, Hq, Hkv, P, d, dtype, fmt):
    x = Batch(prefix, rows, Hq, Hkv, d, P, fmt, dtype, seed=len(prefix) + rows[0])
    x.run()
    x.check()


@pytest.mark.parametrize("splits", [0, 1, 2, 3, 7])
@pytest.mark.parametrize("prefix,rows,Hq,Hkv,P,d", [
    ([2100], [300], 2, 2, 64, 128),                 # two tiles of rows over many tiles of keys
    ([1900], [270], 2, 2, 16, 64),
    ([3000], [17], 2, 1, 32, 128),                  # one tile of rows: the groups take the keys in turn
    ([2305], [5], 8, 1, 48, 64),
    ([0], [1500], 1, 1, 64, 128),                   # new rows only, up to six tiles of rows
    ([700, 0, 1500], [600, 900, 1], 4, 2, 128, 128),
    ([128 * 9, 128 * 8], [256, 128], 1, 1, 64, 128),  # everything whole tiles
])
def test_many_tiles_in_any_number_of_parts(prefix, rows, Hq, Hkv, P, d, splits):
    x = Batch(prefix, rows, Hq, Hkv, d, P, seed=splits)
    ws = x.run(splits=splits)
    x.check()
    first = x.out.clone(), x.lse.clone()
    x.out.fill_(7.0)
    x.run(splits=splits, ws=ws)                     # the workspace is as it was; the same bits again
    assert torch.equal(first[0], x.out) and torch.equal(first[1], x.lse)


@pytest.mark.parametrize("prefix,rows,Hq,Hkv,P,d,unit", [
    ([2000], [700], 64, 8, 64, 128, 256),           # 22 units of 256 rows a KV head
    ([1100, 0, 2300, -1, 40], [260, 600, 130, 9, 1], 64, 16, 32, 64, 256),
    ([3900] * 5, [33] * 5, 32, 32, 16, 128, 256),    # 33 rows a unit
    ([16384], [385], 64, 8, 64, 64, 128),           # 25 units of 128 rows a KV head
])
def test_whole_rounds_of_blocks_and_a_last_one_in_parts(prefix, rows, Hq, Hkv, P, d, unit):
    """As many units as SMs go out whole; what is left over is taken in parts."""
    x = Batch(prefix, rows, Hq, Hkv, d, P, seed=5)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    units = Hkv * ((x.T * (Hq // Hkv) + (unit - 1) * len(rows)) // unit)
    shape = E.ChunkAttnShape(B=len(prefix), rows=x.T, Hq=Hq, max_rows=max(rows), max_blocks=x.table.shape[1])
    S, need = E.et_chunk_attention_paged_splits(shape, x.cache), E.et_chunk_attention_paged_workspace_size(shape, x.cache)
    assert units > sms and S > 1
    assert need == 16384 * 4 + (units % sms) * S * unit * (8 + 4 * d)
    ws = x.run()
    x.check()
    first = x.out.clone(), x.lse.clone()
    x.out.fill_(7.0)
    x.run(ws=ws)
    assert torch.equal(first[0], x.out) and torch.equal(first[1], x.lse)


def test_values_that_are_not_finite_stay_with_the_rows_that_see_them():
    """NaN and infinities in a later row's key or value, in the next sequence's rows and behind the prefix."""
    for dtype in ("bf16", "f32"):
        x = Batch([70, 0], [150, 40], 2, 1, 128, 16, dtype=dtype, seed=3)
        clean = Batch([70, 0], [150, 40], 2, 1, 128, 16, dtype=dtype, seed=3)
        bad_row = 101
        x.v[bad_row, 0, 5] = float("nan")
        x.v[bad_row, 0, 6] = float("inf")
        x.k[140, 0, 7] = float("nan")                 # rows from 140 on score NaN
        x.v[150 + 30, 0, 9] = float("-inf")           # the other sequence's row 30
        x.run()
        clean.run()
        for name in ("out", "lse"):
            a, b = getattr(x, name)[:bad_row], getattr(clean, name)[:bad_row]
            assert torch.equal(a, b)                  # rows before see nothing of it
            assert torch.equal(getattr(x, name)[150:180], getattr(clean, name)[150:180])
        o = x.out[bad_row:140].float()
        assert bool(o[..., 5].isnan().all()) and bool((o[..., 6] == float("inf")).all())
        rest = [d for d in range(128) if d not in (5, 6)]
        assert bool(o[..., rest].isfinite().all())
        assert bool(x.out[140:150].isnan().all())
        tail = x.out[180:190].float()
        assert bool((tail[..., 9] == float("-inf")).all()) and bool(tail[..., :9].isfinite().all())


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_a_query_that_is_not_finite_gives_nan(value):
    for prefix in (0, 200):
        x = Batch([prefix], [20], 4, 2, 64, 32, seed=4)
        x.q[7, 2, 11] = value
        x.run()
        out, lse, mass = x.exact()
        bad = torch.zeros(x.T, 4, dtype=torch.bool, device="cuda")
        bad[7, 2] = True
        assert bool(x.out[bad].isnan().all()) and bool(x.lse[bad].isnan().all())
        err = (x.out.double() - out).abs()[~bad]
        assert bool((err <= 4 * 2.0 ** -9 * (out.abs() + mass)[~bad]).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_indexes_are_reported_and_skipped(dtype):
    # a page id outside the cache drops its tokens
    x = Batch([200], [10], 2, 1, 64, 64, dtype=dtype, seed=5)
    x.table[0, 1] = 10 ** 6
    x.run()
    assert int(x.status.item()) == E.ET_DEV_BAD_INDEX
    keep = torch.cat([torch.arange(64), torch.arange(128, 200)])
    y = Batch([200], [10], 2, 1, 64, 64, dtype=dtype, seed=5)
    pages = y.table[0].long()
    got = x.out
    for h in range(2):
        kk = (y.cache.k_pages.float()[pages, 0] * y.cache.k_scale[pages, 0, None, None]).reshape(-1, 64)[:200][keep].double()
        vv = (y.cache.v_pages.float()[pages, 0] * y.cache.v_scale[pages, 0, None, None]).reshape(-1, 64)[:200][keep].double()
        for i in range(10):
            k = torch.cat([kk, y.k[:i + 1, 0].double()])
            v = torch.cat([vv, y.v[:i + 1, 0].double()])
            p = torch.softmax(k @ y.q[i, h].double() / 8, 0)
            want, mass = p @ v, p @ v.abs()
            assert bool(((got[i, h].double() - want).abs() <= 4 * 2.0 ** -9 * (want.abs() + mass)).all())
    # a prefix past the bound is cut there
    x = Batch([300], [5], 2, 1, 64, 32, dtype=dtype, seed=6)
    x.run(max_prefix=256)
    assert int(x.status.item()) == E.ET_DEV_BAD_INDEX
    x.prefix = [256]
    x.status.zero_()
    x.check()
    # row starts that descend, leave the rows or pass max_rows
    x = Batch([50, 50, 50], [5, 6, 7], 2, 1, 64, 32, dtype=dtype, seed=7)
    out, lse, _ = x.exact()
    x.start[2] = 4                                    # sequence 1 ends before it begins; sequence 2 then has 14 rows of at most 7
    x.run()
    assert int(x.status.item()) == E.ET_DEV_BAD_INDEX
    assert bool(((x.out[:4].double() - out[:4]).abs() <= 0.05 * (1 + out[:4].abs())).all())
    assert bool((x.out[11:] == 7).all())
    x = Batch([50], [5], 2, 1, 64, 32, dtype=dtype, seed=8)
    x.start[1] = x.T + 1
    x.run()
    assert int(x.status.item()) == E.ET_DEV_BAD_INDEX and bool((x.out == 7).all())


@pytest.mark.parametrize("scales", [(-48, -44), (40, 48), (-30, 10)])
def test_scales_far_from_one(scales):
    """V scales far from the new rows' values: what is small on one side is kept as long as fp32 sums hold it."""
    x = Batch([400], [70], 2, 1, 128, 16, seed=9)
    x.cache.v_scale.copy_(2.0 ** torch.randint(scales[0], scales[1] + 1, x.cache.v_scale.shape, device="cuda").float())
    x.run()
    x.check()
    x = Batch([400], [70], 2, 1, 64, 16, seed=10)     # keys whose scale is negative, zero, or no power of two
    x.cache.k_scale.mul_(torch.where(torch.rand(x.cache.k_scale.shape, device="cuda") < 0.3, -1.1, 0.9))
    x.cache.k_scale[x.table[0, 3].long()] = 0.0
    x.run()
    x.check()


def test_queries_of_the_smallest_magnitudes():
    """Rows down to the last subnormal, and zero: every key counts the same, the sum of weights stays right."""
    x = Batch([300, 0], [130, 70], 4, 2, 128, 32, seed=9)
    for i, f in enumerate([0.0, 2.0 ** -133, 2.0 ** -126, 2.0 ** -118, 2.0 ** -117, 2.0 ** -60, 2.0 ** -9, 1.0]):
        x.q[i::8] = (x.q[i::8].float().sign() * f).to(torch.bfloat16) if f < 2.0 ** -100 else x.q[i::8] * f
    x.run()
    x.check()


def test_more_sequences_than_are_ordered():
    """Batches past 32 sequences keep their order; whole units, parts and sequences without rows among them."""
    for n, splits in ((33, 0), (47, 3), (70, 1), (130, 0)):
        prefix = [(37 * b) % 290 - (b % 11 == 5) * 300 for b in range(n)]
        rows = [0 if b % 7 == 3 else 1 + (b * b) % 9 * (40 if b % 13 == 0 else 1) for b in range(n)]
        x = Batch([max(p, -1) for p in prefix], rows, 4, 2, 64, 16, seed=n)
        x.run(splits=splits)
        x.check()


def test_scores_far_apart():
    """Scores that rise by thousands from tile to tile: the reference moves each time; and one row's lie far below another's."""
    x = Batch([1024], [130], 1, 1, 128, 64, seed=11)
    ramp = 2.0 ** (torch.arange(16, device="cuda") / 2)
    x.cache.k_scale[x.table[0].long()] = (ramp * 2.0 ** -8)[:, None]
    x.q[::2] *= 30
    x.run(splits=1)
    out, lse, mass = x.exact()
    # a score of size s carries 2^-24 s of rounding in its sum and product: relative weight errors of 2^-21 s
    slack = 2.0 ** -20 * lse.abs().clamp(min=1)[..., None] * 30
    assert bool(((x.out.double() - out).abs() <= (2 * 2.0 ** -9 + slack) * (out.abs() + mass)).all())
    x.run(splits=4)
    assert bool(((x.out.double() - out).abs() <= (2 * 2.0 ** -9 + slack) * (out.abs() + mass)).all())


def test_graphs_streams_and_one_workspace():
    a, b = Batch([900], [40], 4, 2, 128, 64, seed=12), Batch([500, 600], [3, 90], 2, 1, 64, 32, seed=13)
    sizes = []
    for x in (a, b):
        x.shape = E.ChunkAttnShape(B=len(x.prefix), rows=x.T, Hq=x.Hq, max_rows=max(x.rows), max_blocks=x.table.shape[1],
                                   num_splits=3)
        sizes.append(E.et_chunk_attention_paged_workspace_size(x.shape, x.cache))
    ws = E.new_workspace(max(sizes))

    def call(x, stream=None):
        E.et_chunk_attention_paged(x.shape, x.cache, x.table, x.plen, x.start, x.q, x.k, x.v, x.out, lse=x.lse, ws=ws,
                                   dev_status=x.status, stream=stream)
    for x in (a, b):
        call(x)
    torch.cuda.synchronize()
    graphs = []
    for x in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(x)
        graphs.append(g)
    s = torch.cuda.Stream()
    for lens in ([900], [130], [0]):                  # replayed with other prefixes, the workspace shared in turn
        a.plen.copy_(torch.tensor(lens, dtype=torch.int32))
        a.prefix = lens
        a.out.fill_(7.0)
        a.lse.fill_(7.0)
        torch.cuda.synchronize()
        for g in graphs + graphs:
            g.replay()
        torch.cuda.synchronize()
        a.check()
        b.check()
    b.out.fill_(7.0)
    torch.cuda.synchronize()
    call(b, stream=s)
    s.synchronize()
    b.check()


def test_a_cache_past_32_bits():
    P, Hkv, d = 64, 8, 128
    pages = 40000                                     # 131072 bytes a page, K and V: 5.2 GB
    x = Batch([300], [70], 16, Hkv, d, P, seed=14)
    big = E.PagedCache.allocate(pages, Hkv, P, d)
    old = x.table[0].long().clone()
    new = torch.tensor([pages - 1, 0, pages - 3, 33333, 16500], device="cuda")[:len(old)]
    for src, dst in ((x.cache.k_pages, big.k_pages), (x.cache.v_pages, big.v_pages)):
        for o, n in zip(old.tolist(), new.tolist()):
            dst.view(torch.uint8)[n].copy_(src.view(torch.uint8)[o])
    big.k_scale[new], big.v_scale[new] = x.cache.k_scale[old], x.cache.v_scale[old]
    x.table[0] = new.to(torch.int32)
    x.cache = big
    x.run()
    x.check()


@pytest.mark.parametrize("splits", [1, 3])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(splits):
    """With a bound of one cycle a call reports that it gave up, or every wait was met at its first look and it is right."""
    reported = 0
    for prefix, rows in (([700], [300]), ([700], [20]), ([0], [300])):
        x = Batch(prefix, rows, 2, 1, 128, 64, seed=15)
        try:
            E.et_set_wait_limit(1)
            ws = x.run(splits=splits)
        finally:
            E.et_set_wait_limit(0)
        if int(x.status.item()):
            assert int(x.status.item()) == E.ET_DEV_TIMEOUT
            reported += 1
        else:
            x.check()
        x.status.zero_()
        x.run(splits=splits, ws=ws)
        x.check()
    assert reported > 0


def test_a_prompt_on_its_way():
    """Pages, rotation, attention, commit, piece by piece, then one decoded token and a draw: each step against its formula
    on what the steps before left, and the decoding call against this one."""
    Hq, Hkv, d, P, F, V = 4, 2, 128, 32, 256, 500
    g = torch.Generator(device="cuda").manual_seed(77)
    bf = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    lens, B, cols, pool = [100, 37], 2, 8, 20
    cache = E.PagedCache.allocate(pool, Hkv, P, d)
    table = torch.full((B, cols), -1, dtype=torch.int32, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    nblk, free, count = i32(0, 0), torch.arange(pool, dtype=torch.int32, device="cuda"), i32(pool)
    status, plen, done = i32(0), i32(0, 0), [0, 0]
    freq, factor = E.et_rotary_frequencies(d)
    freq = freq.cuda()
    pieces = [(64, 37), (36, 0), (1, 1)]              # the last one is a decoded token of each
    for piece in pieces:
        T = sum(piece)
        starts = [0, piece[0], T]
        qkv = bf(T, Hq + 2 * Hkv, d)
        pos = torch.cat([torch.arange(n, n + m) for n, m in zip(done, piece)]).to(torch.int32).cuda()
        q, k = torch.zeros(T, Hq, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, Hkv, d, dtype=torch.bfloat16, device="cuda")
        E.et_rotary(E.RotaryShape(rows=T, Hq=Hq, Hkv=Hkv, d=d, factor=factor), pos, freq, qkv[:, :Hq], q, k=qkv[:, Hq:Hq + Hkv], k_out=k)
        v = qkv[:, Hq + Hkv:]
        E.et_block_map(E.BlockMapShape(B=B, page_size=P, max_blocks=cols, num_pages=pool), plen, i32(*piece), nblk, table, free,
                       count, dev_status=status)
        out, lse = torch.zeros(T, Hq, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, Hq, device="cuda")
        shape = E.ChunkAttnShape(B=B, rows=T, Hq=Hq, max_rows=max(piece), max_blocks=cols, max_prefix=cols * P)
        ws = E.new_workspace(E.et_chunk_attention_paged_workspace_size(shape, cache))
        E.et_chunk_attention_paged(shape, cache, table, plen, i32(*starts), q, k, v, out, lse=lse, ws=ws, dev_status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        for b in range(B):
            n, r0, r1 = done[b], starts[b], starts[b + 1]
            pages = table[b, :-(-n // P)].long()
            for h in range(Hq):
                held = lambda x, s: (x.float()[pages, h // 2] * s[pages, h // 2, None, None]).reshape(-1, d)[:n].double()  # noqa: E731
                kk = torch.cat([held(cache.k_pages, cache.k_scale), k[r0:r1, h // 2].double()])
                vv = torch.cat([held(cache.v_pages, cache.v_scale), v[r0:r1, h // 2].double()])
                z = q[r0:r1, h].double() @ kk.T / math.sqrt(d)
                z = z.masked_fill(~torch.ones(r1 - r0, n + r1 - r0, dtype=torch.bool, device="cuda").tril(n), -math.inf)
                p = torch.softmax(z, 1)
                want, mass = p @ vv, p @ vv.abs()
                assert bool(((out[r0:r1, h].double() - want).abs() <= 4 * 2.0 ** -9 * (want.abs() + mass)).all())
        if piece == pieces[-1]:                       # the decoding call says the same
            dshape = E.PagedAttnShape(B=B, N=1, Hq=Hq, max_blocks=cols)
            dws = E.new_workspace(E.et_tree_attention_paged_workspace_size(dshape, cache))
            dout, dlse = torch.zeros(B, 1, Hq, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(B, Hq, 1, device="cuda")
            E.et_tree_attention_paged(dshape, cache, table, plen, q.view(B, 1, Hq, d), k.view(B, 1, Hkv, d),
                                      v.reshape(B, 1, Hkv, d).contiguous(), None, dout, lse=dlse, ws=dws, dev_status=status)
            torch.cuda.synchronize()
            assert bool(((dout.view(B, Hq, d).float() - out.float()).abs() <= 0.03).all())
            assert bool(((dlse.view(B, Hq) - lse).abs() <= 2e-5 * (1 + lse.abs())).all())
        # the rows go into the pages; a sequence without new rows appends none
        N = max(piece)
        kt, vt = (torch.zeros(B, N, Hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        for b in range(B):
            kt[b, :piece[b]], vt[b, :piece[b]] = k[starts[b]:starts[b + 1]], v[starts[b]:starts[b + 1]]
        new_len = i32(0, 0)
        E.et_kv_commit_paged(E.PagedCommitShape(B=B, N=N, path_len=0, max_blocks=cols), cache, table, kt, vt,
                             i32(*[m - 1 for m in piece]), None, plen, new_len, dev_status=status)
        plen = new_len
        done = [n + m for n, m in zip(done, piece)]
    torch.cuda.synchronize()
    assert plen.tolist() == done == [101, 38] and int(status.item()) == 0
    feats, head = out.reshape(B, -1)[:, :F].contiguous(), bf(V, F)
    logits = torch.zeros(B, V, device="cuda")
    E.et_lm_head(feats, head, logits)
    tok = i32(-1, -1)
    E.et_sample(logits, torch.rand(B, generator=g, device="cuda"), tok, top_k=i32(5, 1))
    torch.cuda.synchronize()
    best = torch.topk(logits, 5, dim=1).indices
    assert int(tok[0]) in best[0].tolist() and int(tok[1]) == int(best[1, 0])
