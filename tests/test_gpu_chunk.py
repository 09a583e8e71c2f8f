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


@pytest.mark.parametrize("splits", [1, 2, 3, 7])
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
