"""Acceptance whose inputs another stream is still writing: no result is
promised then, but every block of a cluster takes the leader's decision, so
that the walk stays a walk and no block stores into one that has left."""
import numpy as np
import pytest
import torch

from speculative_decoding_eagle_gb300 import binding as E
from speculative_decoding_eagle_gb300 import workloads as W

pytestmark = pytest.mark.gpu


def accepting(B, V, widths, seed=7):
    """A static tree whose children are likely, its target rows and the buffers of et_verify_accept."""
    parent, rank = W.static_shape(widths)
    N, D, k = parent.size, len(widths), max(widths)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    draft = 2.0 * torch.randn(B * N, V, generator=gen, device="cuda")
    rmap = torch.arange(B * N, dtype=torch.int32, device="cuda").view(B, N)
    tb = E.TreeBuffers.allocate_flat(B, N, root_tok=torch.arange(B, dtype=torch.int32, device="cuda"))
    E.et_static_tree(B, V, k, torch.from_numpy(parent).cuda(), torch.from_numpy(rank).cuda(), draft, rmap, tb)
    cfg = E.TreeCfg(B=B, V=V, depth=D, topk=k, m=k, n=N - 1, temperature=0.5)
    out = dict(accept_len=torch.zeros(B, dtype=torch.int32, device="cuda"),
               path=torch.zeros((B, D + 1), dtype=torch.int32, device="cuda"),
               tokens=torch.zeros((B, D + 1), dtype=torch.int32, device="cuda"))
    return cfg, tb, draft, out, E.new_workspace(E.et_tree_workspace_size(cfg)), parent


def check_walks(cfg, tb, out, parent):
    alen, path, toks = (out[k].cpu().numpy() for k in ("accept_len", "path", "tokens"))
    tok = tb.flat_tok.cpu().numpy()
    assert (alen >= 0).all() and (alen <= cfg.depth).all()
    for b in range(cfg.B):
        assert path[b, 0] == 0 and (path[b, alen[b] + 1:] == -1).all()
        for j in range(1, alen[b] + 1):
            assert parent[path[b, j]] == path[b, j - 1] and toks[b, j - 1] == tok[b, path[b, j]]


@pytest.mark.parametrize("B", [8, 16, 32])
def test_uniforms_written_while_the_walk_reads_them(B):
    cfg, tb, draft, out, ws, parent = accepting(B, 32000, (4, 2, 2, 1, 1))
    uniforms = torch.zeros(B, cfg.n + 1, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    writer, reader = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(150):
        with torch.cuda.stream(writer):  # everything accepted, nothing accepted, in turn
            for u in (0.0, 0.9999999, 0.0, 0.9999999):
                uniforms.fill_(u)
        E.et_verify_accept(cfg, E.ET_ACCEPT_STOCH_POINT, tb, draft, out["accept_len"], out["path"], out["tokens"], ws,
                           uniforms=uniforms, dev_status=status, stream=reader)
    torch.cuda.synchronize()
    check_walks(cfg, tb, out, parent)
    for u, deepest in ((0.0, cfg.depth), (0.9999999, 0)):  # and alone it decides as ever
        uniforms.fill_(u)
        E.et_verify_accept(cfg, E.ET_ACCEPT_STOCH_POINT, tb, draft, out["accept_len"], out["path"], out["tokens"], ws,
                           uniforms=uniforms, dev_status=status)
        torch.cuda.synchronize()
        check_walks(cfg, tb, out, parent)
        assert (out["accept_len"] == deepest).all() and int(status.item()) == 0


@pytest.mark.parametrize("B", [1, 4])
def test_uniforms_written_while_draftq_rows_are_decided(B):
    """Rows of a draft-q tree are decided by a cluster each; its blocks test the children one after the other."""
    cfg, tb, draft, out, ws, parent = accepting(B, 32000, (4, 2, 2, 1, 1))
    gen = torch.Generator(device="cuda").manual_seed(3)
    target = draft + torch.randn(draft.shape, generator=gen, device="cuda")
    uniforms = torch.zeros(B, cfg.n + 1, device="cuda")
    call = lambda stream=None: E.et_verify_accept(  # noqa: E731
        cfg, E.ET_ACCEPT_STOCH_DRAFTQ, tb, target, out["accept_len"], out["path"], out["tokens"], ws, draft_logits=draft,
        uniforms=uniforms, stream=stream)
    torch.cuda.synchronize()
    writer, reader = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(150):
        with torch.cuda.stream(writer):
            for u in (0.0, 0.9999999, 0.0, 0.9999999):
                uniforms.fill_(u)
        call(reader)
    torch.cuda.synchronize()
    check_walks(cfg, tb, out, parent)
    uniforms.fill_(0.5)
    call()
    torch.cuda.synchronize()
    check_walks(cfg, tb, out, parent)
