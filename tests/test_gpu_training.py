"""The training-side operators on the GPU against plain fp64 implementations: rotary positions, the sparse attention's
backward pass, the gradient of the indexer's objective, the backward pass of the index scores, and a run of them
together.

Tolerances.  bf16 rounds a value by at most 2^-9 to 2^-8 of itself (half a step), by 2^-8 / sqrt(12) x sqrt(2) rms at
most.  A bf16 gradient is a sum of products whose factors were rounded at most twice (an operand of the product and the
entry's contribution, to bf16 or finer) plus its own rounding: the relative L2 error of three independent roundings
stays below 2^-8 (they make 0.0033 at most; 2^-8 is 0.0039).  fp32 results that are sums
of n fp32 terms with logits off by 2^-20 stay within 1e-5 in relative L2."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

D, DV = 576, 512
SCALE = D ** -0.5
L2_BF16 = 2.0 ** -8
L2_FP32 = 1e-5


@pytest.fixture(scope="module")
def dsa():
    import sparse_attention_long_05_b200 as m
    return m


def _rel(got, want):
    got, want = got.double().cpu(), want.double().cpu()
    assert torch.isfinite(got).all()
    return float((got - want).norm() / want.norm().clamp(min=1e-300))


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _selection(T, S, k, g, kind):
    """[T, k] int32 on the CPU.  causal: the last T positions of S, ascending; holes: unsorted, with -1 between;
    twice: rows named several times; blank: every second token empty."""
    idx = torch.full((T, k), -1, dtype=torch.int32)
    for t in range(T):
        n = min(k, S - T + t + 1)
        if kind == "causal":
            idx[t, :n] = torch.randperm(S - T + t + 1, generator=g)[:n].sort().values.int()
        elif kind == "holes":
            m = int(torch.randint(1, min(k, S) + 1, (1,), generator=g))
            at = torch.randperm(k, generator=g)[:m]
            idx[t, at] = torch.randperm(S, generator=g)[:m].int()
        elif kind == "twice":
            idx[t] = torch.randint(0, min(S, 40 + 5 * t), (k,), generator=g).int()
            if t == 1:
                idx[t] = 3
        elif kind == "blank" and t % 2:
            idx[t, :n] = torch.randperm(S - T + t + 1, generator=g)[:n].int()
        elif kind == "one":
            idx[t, k - 1] = (7 * t) % S
    return idx


def _attention(q, c, idx):
    """fp64 out and lse of the forward, differentiable."""
    on = idx >= 0
    rows = c[idx.clamp(min=0).long()]
    x = torch.einsum("thd,tkd->thk", q, rows) * SCALE
    x = x.masked_fill(~on[:, None], -math.inf)
    lse = torch.logsumexp(x, 2)
    p = torch.where(on[:, None], (x - torch.where(lse.isinf(), 0.0, lse)[..., None]).exp(), 0.0)
    return torch.einsum("thk,tkd->thd", p, rows[..., :DV]), lse, p, rows


def _attention_case(T, S, H, k, kind, seed):
    g = _gen(seed)
    q = torch.randn(T, H, D, generator=g).bfloat16()
    c = torch.randn(S, D, generator=g).bfloat16()
    dout = torch.randn(T, H, DV, generator=g).bfloat16()
    return q, c, _selection(T, S, k, g, kind), dout


def _formula(q, c, idx, out, lse, dout):
    """dq, dc from the definition, with the given out and lse (fp64)."""
    q, c, out, lse, dout = (t.double() for t in (q, c, out, lse, dout))
    on = (idx >= 0)[:, None]
    rows = c[idx.clamp(min=0).long()]
    p = torch.where(on, (torch.einsum("thd,tkd->thk", q, rows) * SCALE - lse[..., None]).exp(), 0.0)
    dp = torch.einsum("thd,tkd->thk", dout, rows[..., :DV])
    ds = SCALE * p * (dp - (dout * out).sum(-1, keepdim=True))
    each = torch.einsum("thk,thd->tkd", ds, q)
    each[..., :DV] += torch.einsum("thk,thd->tkd", p, dout)
    dc = torch.zeros_like(c).index_add_(0, idx.clamp(min=0).long().flatten(), each.flatten(0, 1))
    return torch.einsum("thk,tkd->thd", ds, rows), dc


def _run_attention(dsa, q, c, idx, dout, **kw):
    qd, cd, idxd, dd = (t.cuda() for t in (q, c, idx, dout))
    out, lse = dsa.dsa_sparse_mla_attn(qd, cd, idxd, SCALE)
    dq, dc = dsa.dsa_sparse_mla_attn_backward(qd, cd, idxd, out, lse, dd, SCALE, **kw)
    assert dsa.dsa_get_device_status() == 0
    return out, lse, dq, dc


# the sums of a chunk's rows take two ways, by the mean length of their lists (16): both occur among these
CASES = [(1, 1, 1, 128, "causal"), (1, 300, 128, 128, "causal"), (3, 130, 8, 192, "causal"), (5, 700, 64, 320, "holes"),
         (9, 200, 65, 128, "twice"), (8, 150, 37, 128, "blank"), (4, 50, 128, 256, "one"), (17, 2300, 128, 2048, "causal"),
         (160, 161, 16, 128, "causal"), (6, 900, 128, 576, "holes")]


@pytest.mark.parametrize("T,S,H,k,kind", CASES)
def test_attention_backward(dsa, T, S, H, k, kind):
    q, c, idx, dout = _attention_case(T, S, H, k, kind, 11 * T + S)
    out, lse, dq, dc = _run_attention(dsa, q, c, idx, dout)
    want_q, want_c = _formula(q, c, idx, out.cpu(), lse.cpu(), dout)
    # a single selected key has P = 1 and dP = delta up to the rounding of out: dS is rounding alone, bounded absolutely
    if S == 1 or kind == "one":
        size = SCALE * (dout.double().norm(dim=2).max() * c.double().norm(dim=1).max()) * 2.0 ** -7
        assert (dq.double().cpu() - want_q).abs().max() <= size * c.double().abs().max()
    else:
        assert _rel(dq, want_q) <= L2_BF16
    assert _rel(dc, want_c) <= L2_BF16
    unused = torch.ones(S, dtype=torch.bool)
    unused[idx[idx >= 0].long()] = False
    assert (dc.cpu()[unused] == 0).all()
    assert (dq.cpu()[(idx < 0).all(1)] == 0).all()


def test_attention_backward_matches_autograd(dsa):
    # the formula itself, against automatic differentiation of the forward in fp64
    q, c, idx, dout = _attention_case(5, 260, 24, 192, "holes", 3)
    qd, cd = q.double().requires_grad_(), c.double().requires_grad_()
    out = _attention(qd, cd, idx)[0]
    out.backward(dout.double())
    _, _, dq, dc = _run_attention(dsa, q, c, idx, dout)
    # the forward's out is rounded to bf16 before delta is formed: one rounding more than _formula has
    assert _rel(dq, qd.grad) <= 2 * L2_BF16 and _rel(dc, cd.grad) <= 2 * L2_BF16


def test_attention_backward_is_the_slope(dsa):
    # against differences of the fp64 forward along random directions
    q, c, idx, dout = _attention_case(3, 150, 16, 128, "causal", 5)
    _, _, dq, dc = _run_attention(dsa, q, c, idx, dout)
    g = _gen(6)
    h = 1e-4
    for name, x, dx in (("q", q, dq), ("c", c, dc)):
        v = torch.randn(x.shape, generator=g).double()
        a = {"q": q.double(), "c": c.double()}
        lo, hi = dict(a), dict(a)
        lo[name], hi[name] = a[name] - h * v, a[name] + h * v
        slope = ((_attention(hi["q"], hi["c"], idx)[0] - _attention(lo["q"], lo["c"], idx)[0]) * dout.double()).sum() / (2 * h)
        got = (dx.double().cpu() * v).sum()
        # the error of the projection: the gradient's relative L2 error times its norm (v is unit normal), five sigma
        assert abs(got - slope) <= 5 * 2 * L2_BF16 * dx.double().norm().cpu()


def test_attention_backward_in_chunks_and_repeated(dsa):
    # more tokens than one chunk holds, over many rows; repeated calls agree bit for bit and reuse a workspace
    T, S, H, k = 300, 70001, 16, 2048
    g = _gen(8)
    q = torch.randn(T, H, D, generator=g).bfloat16().cuda()
    c = torch.randn(S, D, generator=g).bfloat16().cuda()
    dout = torch.randn(T, H, DV, generator=g).bfloat16().cuda()
    idx = torch.randint(0, S, (T, k), generator=g).int().cuda()
    idx[:, 0] = 5                                        # one row that every token selects
    out, lse = dsa.dsa_sparse_mla_attn(q, c, idx, SCALE)
    need = dsa.dsa_sparse_mla_attn_backward_workspace_size(T, S, H, k)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    dq, dc = dsa.dsa_sparse_mla_attn_backward(q, c, idx, out, lse, dout, SCALE, ws=ws)
    ws.fill_(0xab)
    dq2, dc2 = dsa.dsa_sparse_mla_attn_backward(q, c, idx, out, lse, dout, SCALE, ws=ws)
    assert torch.equal(dq, dq2) and torch.equal(dc, dc2)
    assert dsa.dsa_get_device_status() == 0
    want_q, want_c = torch.empty(T, H, D, dtype=torch.float64), torch.zeros(S, D, dtype=torch.float64, device="cuda")
    for a in range(0, T, 50):
        b = slice(a, a + 50)
        x, y = _formula(q[b], c, idx[b], out[b], lse[b], dout[b])
        want_q[b] = x.cpu()
        want_c += y
    assert _rel(dq, want_q) <= L2_BF16 and _rel(dc, want_c) <= L2_BF16


def test_more_tokens_than_a_chunk(dsa):
    # a chunk holds at most 2048 tokens; the last one is shorter, and rows get entries from both
    T, S, k = 2100, 700, 128
    g = _gen(15)
    idx = torch.stack([torch.randperm(S, generator=g)[:k] for _ in range(T)]).int()
    idx[:, 100:] = -1
    idx[2090:, 0] = 7
    q, c = torch.randn(T, 3, D, generator=g).bfloat16().cuda(), torch.randn(S, D, generator=g).bfloat16().cuda()
    dout, idx = torch.randn(T, 3, DV, generator=g).bfloat16().cuda(), idx.cuda()
    out, lse = dsa.dsa_sparse_mla_attn(q, c, idx, SCALE)
    dq, dc = dsa.dsa_sparse_mla_attn_backward(q, c, idx, out, lse, dout, SCALE)
    want_q, want_c = _formula(q, c, idx, out, lse, dout)
    assert _rel(dq, want_q) <= L2_BF16 and _rel(dc, want_c) <= L2_BF16
    qi = torch.randn(T, 4, 64, generator=g).to(torch.float8_e4m3fn).cuda()
    ki = torch.randn(S, 64, generator=g).to(torch.float8_e4m3fn).cuda()
    w, dsel = torch.randn(T, 4, generator=g).cuda(), torch.randn(T, k, generator=g).cuda()
    got = dsa.dsa_indexer_scores_backward(qi, None, ki, None, w, idx, dsel)
    assert dsa.dsa_get_device_status() == 0
    qf, kf, wf = (t.float().double().requires_grad_() for t in (qi, ki, w))
    (_indexer_scores(qf, kf, wf, idx) * torch.where(idx >= 0, dsel.double(), 0.0)).sum().backward()
    assert _rel(got[0], qf.grad) <= L2_BF16 and _rel(got[1], kf.grad) <= L2_BF16 and _rel(got[2], wf.grad) <= L2_FP32


def test_rows_behind_32_bit_offsets(dsa):
    # 4.0 million rows: c and dc hold 2.3e9 elements each, k_idx and dk 5.1e8 (bytes: 4.6e9, 1.0e9)
    T, S, k, H = 2, 4_000_000, 128, 4
    g = _gen(16)
    near = torch.randint(0, 1000, (T, 64), generator=g)
    idx = torch.cat([near.sort(1).values.unique(dim=1)[:, :32], S - 1 - torch.arange(96).expand(T, 96)], 1).int().cuda()
    assert idx.shape == (T, k)
    rows = idx.long().unique()
    c = torch.zeros(S, D, dtype=torch.bfloat16, device="cuda")
    c[rows] = torch.randn(len(rows), D, generator=g).bfloat16().cuda()
    q, dout = (torch.randn(T, H, n, generator=g).bfloat16().cuda() for n in (D, DV))
    out, lse = dsa.dsa_sparse_mla_attn(q, c, idx, SCALE)
    dq, dc = dsa.dsa_sparse_mla_attn_backward(q, c, idx, out, lse, dout, SCALE)
    assert dsa.dsa_get_device_status() == 0
    where = torch.searchsorted(rows, idx.long()).int()
    want_q, want_c = _formula(q, c[rows], where, out, lse, dout)
    assert _rel(dq, want_q) <= L2_BF16 and _rel(dc[rows], want_c) <= L2_BF16
    dc[rows] = 0
    assert not dc.any()
    del c, dc
    ki = torch.zeros(S, 128, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    ki.view(torch.uint8)[rows] = torch.randn(len(rows), 128, generator=g).to(torch.float8_e4m3fn).view(torch.uint8).cuda()
    qi = torch.randn(T, 64, 128, generator=g).to(torch.float8_e4m3fn).cuda()
    w, dsel = torch.randn(T, 64, generator=g).cuda(), torch.randn(T, k, generator=g).cuda()
    got = dsa.dsa_indexer_scores_backward(qi, None, ki, None, w, idx, dsel)
    qf, kf, wf = (t.float().double().requires_grad_() for t in (qi, ki.view(torch.uint8)[rows].view(torch.float8_e4m3fn), w))
    (_indexer_scores(qf, kf, wf, where) * dsel.double()).sum().backward()
    assert _rel(got[0], qf.grad) <= L2_BF16 and _rel(got[1][rows], kf.grad) <= L2_BF16 and _rel(got[2], wf.grad) <= L2_FP32


def test_attention_backward_nan_rows_nobody_selects(dsa):
    q, c, idx, dout = _attention_case(6, 400, 20, 192, "holes", 9)
    used = torch.zeros(400, dtype=torch.bool)
    used[idx[idx >= 0].long()] = True
    idx[2] = -1                                          # an empty token with NaN queries
    clean = _run_attention(dsa, q, c, idx, dout)
    c2, q2 = c.clone(), q.clone()
    used = torch.zeros(400, dtype=torch.bool)
    used[idx[idx >= 0].long()] = True
    c2[~used] = math.nan
    q2[2] = math.nan
    out, lse = (t.cuda() for t in (clean[0].cpu(), clean[1].cpu()))
    dq, dc = dsa.dsa_sparse_mla_attn_backward(q2.cuda(), c2.cuda(), idx.cuda(), out, lse, dout.cuda(), SCALE)
    assert torch.equal(dq, clean[2]) and torch.equal(dc, clean[3])


@pytest.mark.parametrize("size", [2.0 ** -100, 2.0 ** -40, 2.0 ** 60, 2.0 ** 100])
def test_gradients_scale_with_their_input(dsa, size):
    # a power of two moves through every rounding of the pass: P is the same, all else scales exactly
    q, c, idx, dout = _attention_case(5, 300, 24, 192, "holes", 4)
    out, lse, dq, dc = _run_attention(dsa, q, c, idx, dout)
    dq2, dc2 = dsa.dsa_sparse_mla_attn_backward(q.cuda(), c.cuda(), idx.cuda(), out, lse, (dout * size).cuda(), SCALE)
    assert torch.equal(dq2.double(), dq.double() * size) and torch.equal(dc2.double(), dc.double() * size)
    qi, qs, kk, ks, w, idx, dsel = _indexer_case(5, 300, 64, 128, 192, "holes", True, 6)
    dev = [t.cuda() for t in (qi, qs, kk, ks, w, idx)]
    a = dsa.dsa_indexer_scores_backward(*dev, dsel.cuda())
    b = dsa.dsa_indexer_scores_backward(*dev, (dsel * size).cuda())
    # G q_scale and G k_scale are bf16 operands, whose subnormals the tensor cores may take as zero: each is then off by at
    # most 2^-126, and an element of dq or dk by that times 448 (the largest e4m3) for each of at most 64 x 192 terms.
    # Only the smallest size meets this: there the rms of G k_scale is 2^-100 x 2^-7.6 (dsel) x 2^-6.9 (k_scale) x 2^-3 (w) =
    # 2^-117.5, against which 2^-126 is 2^-8.5 in relative L2.
    for x, y in zip(a, b):
        assert ((y.double() - x.double() * size).abs() <= 64 * 192 * 448 * 2.0 ** -126).all()
        assert _rel(y.double() / size, x) <= L2_BF16


def test_infinite_gradients_reach_what_they_touch(dsa):
    q, c, idx, dout = _attention_case(4, 300, 16, 128, "causal", 13)
    out, lse, dq, dc = _run_attention(dsa, q, c, idx, dout)
    dout[1, 3, 7] = math.inf
    dq2, dc2 = dsa.dsa_sparse_mla_attn_backward(q.cuda(), c.cuda(), idx.cuda(), out, lse, dout.cuda(), SCALE)
    hit = torch.zeros(300, dtype=torch.bool)
    hit[idx[1].long()] = True
    assert not torch.isfinite(dc2.cpu()[hit]).all(1).any() and torch.equal(dc2.cpu()[~hit], dc.cpu()[~hit])
    same = torch.ones(4, 16, dtype=torch.bool)
    same[1, 3] = False
    assert torch.equal(dq2.cpu()[same], dq.cpu()[same]) and not torch.isfinite(dq2.cpu()[1, 3]).any()


@pytest.mark.parametrize("T,S,H,k", [(64, 600, 16, 320), (24, 24000, 16, 320)])    # long lists, short lists
def test_gradients_are_not_biased(dsa, T, S, H, k):
    """sum(got want) / sum(want^2) - 1: roundings that go up as often as down leave 2^-8 / sqrt(n) of it, n = T k H or more
    independent ones (1.2e-5 at most here); cutting each contribution off at ten bits leaves -3.5e-4."""
    def shift(got, want):
        got, want = got.double().cpu(), want.double().cpu()
        return float((got * want).sum() / (want * want).sum()) - 1

    q, c, idx, dout = _attention_case(T, S, H, k, "causal", 2 * T)
    out, lse, dq, dc = _run_attention(dsa, q, c, idx, dout)
    want_q, want_c = _formula(q, c, idx, out.cpu(), lse.cpu(), dout)
    assert abs(shift(dq, want_q)) <= 1e-4 and abs(shift(dc, want_c)) <= 1e-4
    for scaled in (True, False):
        qi, qs, kk, ks, w, idx, dsel = _indexer_case(T, S, 64, 128, k, "causal", scaled, 3 * T)
        dq, dk, dw = dsa.dsa_indexer_scores_backward(*[None if t is None else t.cuda() for t in (qi, qs, kk, ks, w, idx, dsel)])
        qf, kf = qi.float().double(), kk.float().double()
        if scaled:
            qf, kf = qf * qs.double()[:, None, None], kf * ks.double()[:, None]
        qf, kf, wf = qf.requires_grad_(), kf.requires_grad_(), w.double().requires_grad_()
        (_indexer_scores(qf, kf, wf, idx) * torch.where(idx >= 0, dsel.double(), 0.0)).sum().backward()
        assert max(abs(shift(dq, qf.grad)), abs(shift(dk, kf.grad)), abs(shift(dw, wf.grad))) <= 1e-4


@pytest.mark.parametrize("S", [2, 200])                  # the sums of long and of short lists
def test_values_beside_an_infinity_are_kept(dsa, S):
    """A contribution that overflows fp32 in one dim is finite, and exact, in the dims beside it: powers of two, with two
    keys of equal weight."""
    q, c, dout = torch.zeros(1, 1, D), torch.zeros(S, D), torch.zeros(1, 1, DV)
    q[0, 0, 5], q[0, 0, 7] = 2.0 ** 13, 1.0              # the keys are 0 there: both logits are 0, P = 1/2
    c[0, 0], c[1, 0] = 1.0, -1.0
    dout[0, 0, 0] = 2.0 ** 118                           # dP = 2^118 and its negative, delta = 0, dS = scale / 2 of that
    idx = torch.full((1, 128), -1, dtype=torch.int32)
    idx[0, :2] = torch.tensor([0, 1])
    want = torch.zeros(S, D)
    want[0, 0], want[0, 7], want[0, 5] = 2.0 ** 117, 2.0 ** 116, math.inf
    want[1, 0], want[1, 7], want[1, 5] = 2.0 ** 117, -2.0 ** 116, -math.inf
    qd, cd, dd = (t.bfloat16().cuda() for t in (q, c, dout))
    out, lse = dsa.dsa_sparse_mla_attn(qd, cd, idx.cuda(), 0.5)
    _, dc = dsa.dsa_sparse_mla_attn_backward(qd, cd, idx.cuda(), out, lse, dd, 0.5)
    # P, dS and the result are rounded to bf16: 2^-8 of a value at most, each
    fin = want.isfinite()
    assert ((dc.float().cpu() - want)[fin].abs() <= want[fin].abs() * 3 * 2.0 ** -8).all()
    assert torch.equal(dc.float().cpu()[~fin], want[~fin])
    # index scores: one live head, whose query has one large dim
    qi, ki, w = torch.zeros(1, 4, 64), torch.zeros(S, 64), torch.zeros(1, 4)
    qi[0, 0], qi[0, 0, 5], ki[0], w[0, 0] = 1.0, 448.0, 1.0, 1.0
    sel = torch.zeros(1, 128)
    sel[0, 0] = 2.0 ** 120
    idx[0, 1] = -1
    dq, dk, _ = dsa.dsa_indexer_scores_backward(qi.to(torch.float8_e4m3fn).cuda(), None, ki.to(torch.float8_e4m3fn).cuda(),
                                                None, w.cuda(), idx.cuda(), sel.cuda())
    want = torch.zeros(S, 64)
    want[0], want[0, 5] = 2.0 ** 120, math.inf
    assert torch.equal(dk.float().cpu(), want) and (dq[0, 0].float() == 2.0 ** 120).all()
    assert dsa.dsa_get_device_status() == 0


def test_bad_indices_are_recorded_and_skipped(dsa):
    q, c, idx, dout = _attention_case(4, 300, 16, 128, "causal", 12)
    _, _, dq, dc = _run_attention(dsa, q, c, idx, dout)
    out, lse = dsa.dsa_sparse_mla_attn(q.cuda(), c.cuda(), idx.cuda(), SCALE)
    bad = torch.cat([idx, torch.full((4, 64), -1, dtype=torch.int32)], 1)
    bad[0, 130], bad[2, 140], bad[3, 150] = 300, -2, 2 ** 31 - 1
    dq2, dc2 = dsa.dsa_sparse_mla_attn_backward(q.cuda(), c.cuda(), bad.cuda(), out, lse, dout.cuda(), SCALE)
    assert dsa.dsa_get_device_status() == 6             # DSA_ERR_BAD_INDEX
    assert torch.equal(dq, dq2) and torch.equal(dc, dc2)


# ------------------------------------------------------------------------------------------------ indexer objective
@pytest.mark.parametrize("T,S,H,k,kind", CASES)
def test_objective_backward(dsa, T, S, H, k, kind):
    q, c, idx, _ = _attention_case(T, S, H, k, kind, 5 * T + S)
    g = _gen(T)
    sel, dkl = 3 * torch.randn(T, k, generator=g), torch.randn(T, generator=g)
    qd, cd, idxd = q.cuda(), c.cuda(), idx.cuda()
    _, lse = dsa.dsa_sparse_mla_attn(qd, cd, idxd, SCALE)
    got = dsa.dsa_indexer_kl_backward(qd, cd, idxd, sel.cuda(), lse, dkl.cuda(), SCALE)
    assert dsa.dsa_get_device_status() == 0
    _, _, p, _ = _attention(q.double(), c.double(), idx)
    target = p.sum(1)
    target = target / target.sum(1, keepdim=True).clamp(min=1e-300)
    x = sel.double().requires_grad_()
    on = idx >= 0
    logq = torch.log_softmax(x.masked_fill(~on, -1e300), 1)
    kl = torch.where(on & (target > 0), target * (target.clamp(min=1e-300).log() - logq), 0.0).sum(1)
    kl.backward(dkl.double())
    want = torch.where(on, x.grad, 0.0)
    if kind == "one" or S == 1:
        assert (got == 0).all()                          # both distributions are the one entry, exactly
    else:
        assert _rel(got, want) <= L2_FP32
    assert (got.cpu()[~on] == 0).all()
    # without a gradient of the divergences every token counts once
    ones = dsa.dsa_indexer_kl_backward(qd, cd, idxd, sel.cuda(), lse, None, SCALE)
    assert torch.equal(ones, dsa.dsa_indexer_kl_backward(qd, cd, idxd, sel.cuda(), lse, torch.ones(T, device="cuda"), SCALE))


def test_objective_backward_with_nan_and_infinite_scores(dsa):
    """Softmax(I) - p of a token with a NaN among its selected scores is NaN, whichever slot (and so whichever lane, warp or
    CTA of the pair) holds it; a NaN in an empty slot is not looked at; a score of -inf has a softmax of 0."""
    T, S, H, k = 9, 900, 24, 640
    q, c, idx, _ = _attention_case(T, S, H, k, "causal", 17)
    idx[2, 100:], idx[6, 1:], idx[8] = -1, -1, -1
    g = _gen(18)
    sel, dkl = torch.randn(T, k, generator=g), torch.randn(T, generator=g)
    qd, cd, idxd = q.cuda(), c.cuda(), idx.cuda()
    _, lse = dsa.dsa_sparse_mla_attn(qd, cd, idxd, SCALE)
    run = lambda x: dsa.dsa_indexer_kl_backward(qd, cd, idxd, x.cuda(), lse, dkl.cuda(), SCALE)
    clean = run(sel)
    bad = sel.clone()
    bad[2, 100:], bad[8] = math.nan, math.nan            # empty slots only
    bad[1, 0], bad[3, 130], bad[4, 639], bad[5], bad[6, 0] = math.nan, math.nan, math.nan, math.nan, math.nan
    bad[7, 5:300] = -math.inf
    got, on = run(bad).cpu(), idx >= 0
    hit = torch.zeros(T, dtype=torch.bool)
    hit[[1, 3, 4, 5, 6]] = True
    assert torch.isnan(got[hit][on[hit]]).all() and (got[~on] == 0).all()
    same = ~hit
    same[7] = False
    assert torch.equal(got[same], clean.cpu()[same])
    _, _, p, _ = _attention(q.double(), c.double(), idx)
    want = dkl.double()[7] * (torch.softmax(bad[7].double(), 0) - p[7].sum(0) / p[7].sum())
    assert _rel(got[7], want) <= L2_FP32
    # every score -inf: no softmax at all, minus the target is left
    bad[7] = -math.inf
    assert _rel(run(bad)[7], -dkl.double()[7] * p[7].sum(0) / p[7].sum()) <= L2_FP32
    assert dsa.dsa_get_device_status() == 0


# ------------------------------------------------------------------------------------------------ index scores
def _indexer_case(T, S, heads, dim, k, kind, scaled, seed):
    g = _gen(seed)
    if scaled:
        q, kk = torch.randn(T, heads, dim, generator=g), torch.randn(S, dim, generator=g)
        qs, ks = q.abs().amax((1, 2)) / 448, kk.abs().amax(1) / 448
        q, kk = (q / qs[:, None, None]).clamp(-448, 448), (kk / ks[:, None]).clamp(-448, 448)
        w = torch.randn(T, heads, generator=g) * heads ** -0.5
    else:
        q = torch.randint(-7, 8, (T, heads, dim), generator=g).float()
        kk = torch.randint(-7, 8, (S, dim), generator=g).float()
        qs = ks = None
        w = torch.randint(-3, 4, (T, heads), generator=g).float()
    idx = _selection(T, S, k, g, kind)
    return q.to(torch.float8_e4m3fn), qs, kk.to(torch.float8_e4m3fn), ks, w, idx, torch.randn(T, k, generator=g) / k


def _indexer_scores(q, k, w, idx):
    x = torch.einsum("thd,tkd->thk", q, k[idx.clamp(min=0).long()]).relu()
    return torch.einsum("th,thk->tk", w, x)


@pytest.mark.parametrize("heads,dim", [(64, 128), (4, 64)])
@pytest.mark.parametrize("T,S,k,kind,scaled", [(1, 1, 128, "causal", False), (3, 130, 192, "causal", True),
                                               (5, 700, 320, "holes", True), (9, 200, 128, "twice", True),
                                               (8, 150, 128, "blank", False), (4, 50, 256, "one", True),
                                               (17, 2300, 2048, "causal", True), (160, 161, 128, "causal", False)])
def test_index_scores_backward(dsa, heads, dim, T, S, k, kind, scaled):
    q, qs, kk, ks, w, idx, dsel = _indexer_case(T, S, heads, dim, k, kind, scaled, 7 * T + S)
    dev = [None if t is None else t.cuda() for t in (q, qs, kk, ks, w, idx, dsel)]
    dq, dk, dw = dsa.dsa_indexer_scores_backward(*dev)
    assert dsa.dsa_get_device_status() == 0
    qf, kf = q.float().double(), kk.float().double()
    if scaled:
        qf, kf = qf * qs.double()[:, None, None], kf * ks.double()[:, None]
    qf, kf, wf = qf.requires_grad_(), kf.requires_grad_(), w.double().requires_grad_()
    on = idx >= 0
    (_indexer_scores(qf, kf, wf, idx) * torch.where(on, dsel.double(), 0.0)).sum().backward()
    assert _rel(dq, qf.grad) <= L2_BF16
    assert _rel(dk, kf.grad) <= L2_BF16
    assert _rel(dw, wf.grad) <= L2_FP32
    unused = torch.ones(S, dtype=torch.bool)
    unused[idx[on].long()] = False
    assert (dk.cpu()[unused] == 0).all()
    again = dsa.dsa_indexer_scores_backward(*dev)
    assert all(torch.equal(a, b) for a, b in zip((dq, dk, dw), again))


@pytest.mark.parametrize("heads,dim", [(64, 128), (4, 64)])
def test_index_scores_backward_of_sums_that_cancel(dsa, heads, dim):
    """The largest products cancel in pairs, one product of 2^-15 of their sum or more decides the sign, and small ones have
    bits below fp32's: the live heads are those of the exact sum."""
    T, S, k = 12, 300, 192
    g = _gen(dim)
    big = dim // 2 - 4
    q, kk = torch.zeros(T, heads, dim), torch.zeros(S, dim)
    q[..., :big] = 224 + 224 * torch.rand(T, heads, big, generator=g)
    kk[:, :big] = (224 + 224 * torch.rand(S, big, generator=g)) * torch.randn(S, big, generator=g).sign()
    q[..., big:2 * big], kk[:, big:2 * big] = q[..., :big], -kk[:, :big]
    for t in (q, kk):
        t[..., 2 * big] = (32 + 416 * torch.rand(t.shape[:-1], generator=g)) * torch.randn(t.shape[:-1], generator=g).sign()
        t[..., 2 * big + 1:] = 2.0 ** -5 * torch.randn(*t.shape[:-1], dim - 2 * big - 1, generator=g)
    q, kk = q.to(torch.float8_e4m3fn), kk.to(torch.float8_e4m3fn)
    qf, kf = q.float().double(), kk.float().double()
    size = torch.einsum("thd,sd->ths", qf.abs(), kf.abs())
    assert (torch.einsum("thd,sd->ths", qf, kf).abs() >= 2.0 ** -15 * size).all() and size.max() > 2.0 ** 20
    w, idx = torch.randn(T, heads, generator=g), _selection(T, S, k, g, "holes")
    dsel = torch.randn(T, k, generator=g)
    dq, dk, dw = dsa.dsa_indexer_scores_backward(q.cuda(), None, kk.cuda(), None, w.cuda(), idx.cuda(), dsel.cuda())
    assert dsa.dsa_get_device_status() == 0
    qf, kf, wf = qf.requires_grad_(), kf.requires_grad_(), w.double().requires_grad_()
    (_indexer_scores(qf, kf, wf, idx) * torch.where(idx >= 0, dsel.double(), 0.0)).sum().backward()
    assert _rel(dq, qf.grad) <= L2_BF16 and _rel(dk, kf.grad) <= L2_BF16
    # dw takes x itself, which is off by 2^-15 of sum |q k| at most; each live entry's error adds up
    bound = 2.0 ** -15 * torch.einsum("tk,thk->th", torch.where(idx >= 0, dsel.abs().double(), 0.0),
                                      size.gather(2, idx.clamp(min=0).long()[:, None].expand(-1, heads, -1)))
    assert ((dw.double().cpu() - wf.grad).abs() <= bound).all()


def _shifted(t):
    """The same fp32 values in memory that is aligned to 4 bytes only."""
    at = torch.empty(t.numel() + 1, device="cuda")[1:].view(t.shape)
    assert at.data_ptr() % 16 == 4
    return at.copy_(t)


def test_fp32_arrays_at_any_address(dsa):
    """fp32 arguments need the alignment of their type, no more: few tokens (whose items are split and joined) and many
    give the same bits from arrays that start 4 bytes behind a 16-byte boundary."""
    for heads, dim in ((64, 128), (4, 64)):
        for T in (3, 400):
            case = _indexer_case(T, 700, heads, dim, 640, "causal", True, 11 + T)
            q, qs, kk, ks, w, idx, dsel = (t.cuda() for t in case)
            want = dsa.dsa_indexer_scores_backward(q, qs, kk, ks, w, idx, dsel)
            dw = _shifted(torch.zeros_like(w))
            got = dsa.dsa_indexer_scores_backward(q, _shifted(qs), kk, _shifted(ks), _shifted(w), idx, _shifted(dsel),
                                                  dw=dw)
            assert all(torch.equal(a, b) for a, b in zip(got, want))
    for T in (3, 200):
        q, c, idx, dout = (t.cuda() for t in _attention_case(T, 700, 128, 640, "causal", 13 + T))
        out, lse = dsa.dsa_sparse_mla_attn(q, c, idx, SCALE)[:2]
        want = dsa.dsa_sparse_mla_attn_backward(q, c, idx, out, lse, dout, SCALE)
        got = dsa.dsa_sparse_mla_attn_backward(q, c, idx, out, _shifted(lse), dout, SCALE)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        sel, dkl = torch.randn(T, 640, device="cuda"), torch.randn(T, device="cuda")
        want = dsa.dsa_indexer_kl_backward(q, c, idx, sel, lse, dkl, SCALE)
        got = dsa.dsa_indexer_kl_backward(q, c, idx, _shifted(sel), _shifted(lse), _shifted(dkl), SCALE,
                                          dsel=_shifted(torch.zeros_like(sel)))
        assert torch.equal(got, want)


@pytest.mark.parametrize("off", [16, 48, 240])
def test_workspaces_at_any_16_bytes(dsa, off):
    """A workspace of just the stated size, `off` bytes behind a 256-byte boundary: the same bits as one on it, and
    nothing written before or behind it."""
    def workspace(need):
        buf = torch.full((need + 512,), 0xab, dtype=torch.uint8, device="cuda")
        assert buf.data_ptr() % 256 == 0
        return buf, buf[off:off + need]

    def untouched(buf, need):
        return bool((buf[:off] == 0xab).all()) and bool((buf[off + need:] == 0xab).all())

    for T, S, H, k in ((3, 500, 128, 320), (40, 700, 24, 192), (200, 700, 128, 640)):
        q, c, idx, dout = (t.cuda() for t in _attention_case(T, S, H, k, "causal", 3 * T))
        out, lse = dsa.dsa_sparse_mla_attn(q, c, idx, SCALE)
        need = dsa.dsa_sparse_mla_attn_backward_workspace_size(T, S, H, k)
        buf, ws = workspace(need)
        want = dsa.dsa_sparse_mla_attn_backward(q, c, idx, out, lse, dout, SCALE)
        got = dsa.dsa_sparse_mla_attn_backward(q, c, idx, out, lse, dout, SCALE, ws=ws)
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and untouched(buf, need)
        sel = torch.randn(T, k, generator=_gen(T)).cuda()
        need = dsa.dsa_indexer_kl_backward_workspace_size(T)
        buf, ws = workspace(need)
        want = dsa.dsa_indexer_kl_backward(q, c, idx, sel, lse, None, SCALE)
        assert torch.equal(dsa.dsa_indexer_kl_backward(q, c, idx, sel, lse, None, SCALE, ws=ws), want)
        assert untouched(buf, need)
        for heads, dim in ((64, 128), (4, 64)):
            case = [t.cuda() for t in _indexer_case(T, S, heads, dim, k, "causal", True, T)]
            need = dsa.dsa_indexer_scores_backward_workspace_size(T, S, heads, dim, k)
            buf, ws = workspace(need)
            want = dsa.dsa_indexer_scores_backward(*case)
            got = dsa.dsa_indexer_scores_backward(*case, ws=ws)
            assert all(torch.equal(a, b) for a, b in zip(got, want)) and untouched(buf, need)
    assert dsa.dsa_get_device_status() == 0


def test_index_scores_backward_is_the_slope_of_the_forward(dsa):
    # dw against the forward kernel itself: the scores are linear in w
    q, qs, kk, ks, w, idx, dsel = _indexer_case(6, 500, 64, 128, 192, "causal", True, 4)
    dev = [t.cuda() for t in (q, qs, kk, ks, w, idx, dsel)]
    _, _, dw = dsa.dsa_indexer_scores_backward(*dev)
    v = torch.randn(w.shape, generator=_gen(5)).cuda()
    scores = dsa.dsa_indexer_scores(dev[0], dev[1], dev[2], dev[3], v, pos0=500)
    up = torch.where(dev[5] >= 0, scores.gather(1, dev[5].clamp(min=0).long()) * dev[6], 0.0).double().sum()
    size = (scores.abs().max() * dev[6].abs().sum()).item()
    assert abs(float((dw.double() * v.double()).sum() - up)) <= 1e-6 * size


# ------------------------------------------------------------------------------------------------ rotary positions
def _rope_reference(x, f, pos, off, inter, m, backward):
    y = x.double().clone()
    R = 2 * len(f)
    theta = pos.double()[:, None] * f.double()[None]
    cos, sin = m * theta.cos()[:, None], m * theta.sin()[:, None] * (-1 if backward else 1)
    a, b = (slice(off, off + R, 2), slice(off + 1, off + R, 2)) if inter else (slice(off, off + R // 2), slice(off + R // 2, off + R))
    y[..., a], y[..., b] = x.double()[..., a] * cos - x.double()[..., b] * sin, x.double()[..., a] * sin + x.double()[..., b] * cos
    return y


def _rope_close(got, want, x, m):
    # half a step of the type, plus the angle's fp32 sine (2^-20 for bf16, 2^-22 for fp32) times the pair's size
    eps = torch.finfo(got.dtype).eps / 2
    slack = (2.0 ** -20 if got.dtype == torch.bfloat16 else 2.0 ** -21) * 2 * m * float(x.abs().max())
    err = (got.double().cpu() - want).abs()
    assert bool((err <= want.abs() * eps * (1 + 2.0 ** -6) + slack).all()), float(err.max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [True, False])
@pytest.mark.parametrize("T,H,D,R,off", [(1, 1, 64, 64, 0), (3, 128, 576, 64, 512), (7, 5, 128, 64, 0), (130, 1, 72, 16, 8),
                                         (2, 3, 11, 6, 3), (33, 64, 128, 128, 0), (5, 2, 96, 24, 40)])
def test_rope(dsa, dtype, inter, T, H, D, R, off):
    g = _gen(T + D)
    x = torch.randn(T, H, D, generator=g).to(dtype)
    pos = torch.randint(0, 1_000_000, (T,), generator=g, dtype=torch.int32)
    f, m = dsa.dsa_rope_frequencies(R, 10000.0, factor=8.0, orig_len=4096)
    fd, xd, pd = f.cuda(), x.cuda(), pos.cuda()
    y = dsa.dsa_rope(xd, fd, pd, rot_off=off, interleaved=inter, mscale=m)
    assert torch.equal(xd.cpu(), x)
    want = _rope_reference(x, f, pos, off, inter, m, False)
    _rope_close(y, want, x, m)
    keep = [d for d in range(D) if not off <= d < off + R]
    assert torch.equal(y.cpu()[..., keep], x[..., keep])
    # in place, and the gradient: the transpose
    inpl = xd.clone()
    assert dsa.dsa_rope(inpl, fd, pd, rot_off=off, interleaved=inter, mscale=m, out=inpl) is inpl
    assert torch.equal(inpl, y)
    back = dsa.dsa_rope_backward(xd, fd, pd, rot_off=off, interleaved=inter, mscale=m)
    _rope_close(back, _rope_reference(x, f, pos, off, inter, m, True), x, m)


def test_rope_strides_offsets_and_positions(dsa):
    g = _gen(1)
    f = dsa.dsa_rope_frequencies(64)[0].cuda()
    wide = torch.randn(20, 8, 576, generator=g).bfloat16().cuda()
    q = wide[:, :, 512:]                                                     # the position dims of wider rows
    want = _rope_reference(q.cpu(), f.cpu(), torch.arange(20) + 90, 0, True, 1.0, False)
    _rope_close(dsa.dsa_rope(q, f, pos0=90), want, q.cpu(), 1.0)
    flipped = wide.transpose(0, 1)[:, :, 512:]                               # heads outermost
    pos = torch.arange(8, dtype=torch.int32, device="cuda") * 1000
    got = dsa.dsa_rope(flipped, f, pos)
    _rope_close(got, _rope_reference(flipped.cpu(), f.cpu(), pos.cpu(), 0, True, 1.0, False), wide.cpu(), 1.0)
    odd = torch.randn(9, 3, 67, generator=g).bfloat16().cuda()[:, :, 1:65]   # rows that no 16-byte piece fits
    _rope_close(dsa.dsa_rope(odd, f, pos0=5, interleaved=False),
                _rope_reference(odd.cpu(), f.cpu(), torch.arange(9) + 5, 0, False, 1.0, False), odd.cpu(), 1.0)
    # in place on a view: the rest of the rows stays
    before = wide.clone()
    dsa.dsa_rope(q, f, pos0=90, out=q)
    assert torch.equal(wide[..., :512], before[..., :512])
    _rope_close(q, want, before.cpu(), 1.0)
    # positions before the first, and both ends of their range
    ends = torch.tensor([-1, -1000, -2 ** 31, 2 ** 31 - 1, 0], dtype=torch.int32)
    x = torch.randn(5, 2, 64, generator=g)
    _rope_close(dsa.dsa_rope(x.cuda(), f, ends.cuda()), _rope_reference(x, f.cpu(), ends, 0, True, 1.0, False), x, 1.0)
    # into the gaps of the same buffer
    both = torch.randn(6, 1, 128, generator=g).cuda()
    x, out = both[..., :64], both[..., 64:]
    keep = x.clone()
    dsa.dsa_rope(x, f, pos0=3, out=out)
    assert torch.equal(x, keep)
    _rope_close(out, _rope_reference(keep.cpu(), f.cpu(), torch.arange(6) + 3, 0, True, 1.0, False), keep.cpu(), 1.0)
    # one input row for every token
    row = torch.randn(1, 4, 64, generator=g).cuda().expand(5, 4, 64)
    _rope_close(dsa.dsa_rope(row, f), _rope_reference(row.cpu(), f.cpu(), torch.arange(5), 0, True, 1.0, False), row.cpu(), 1.0)
    assert dsa.dsa_rope(both[:0], f).shape == (0, 1, 128)


def test_rope_angles_at_any_position(dsa):
    """Pairs (1, 0) turn to (cos, sin): angles against exact arithmetic.  Bound: 2^-24 turns, |position| f 2^-54 turns, and
    2^-22 for sine, cosine and the result in fp32 (a few units of 2^-24 each)."""
    from decimal import Decimal, getcontext
    getcontext().prec = 60
    pi = Decimal("3.14159265358979323846264338327950288419716939937510582097494")
    pos = [0, 1, -1, 4095, 131071, 10 ** 6 + 1, 2 ** 24 + 1, -(2 ** 24) - 3, 10 ** 8 + 7, 2 ** 31 - 1, -2 ** 31]
    f = torch.cat([dsa.dsa_rope_frequencies(32)[0], torch.tensor([2.5, 0.5, 1e-9, 3.0], dtype=torch.float64)])
    x = torch.tensor([1.0, 0.0]).repeat(len(f)).expand(len(pos), 1, -1).contiguous().cuda()
    y = dsa.dsa_rope(x, f.cuda(), torch.tensor(pos, dtype=torch.int64).int().cuda()).cpu().double()
    for t, p in enumerate(pos):
        for i, w in enumerate(f.tolist()):
            turns = p * Decimal(w) / (2 * pi)
            angle = float((turns - turns.to_integral_value()) * 2 * pi)
            bound = 2 * math.pi * (2.0 ** -24 + abs(p) * w * 2.0 ** -54) + 2.0 ** -22
            assert abs(float(y[t, 0, 2 * i]) - math.cos(angle)) <= bound, (p, w)
            assert abs(float(y[t, 0, 2 * i + 1]) - math.sin(angle)) <= bound, (p, w)


@pytest.mark.parametrize("shape,at", [((5, 3, 4, 64), 1), ((5, 4, 3, 64), 2), ((4, 5, 3, 64), 2), ((3, 4, 5, 64), 0)])
@pytest.mark.parametrize("swap", [False, True])
def test_rope_between_parts_of_one_array(dsa, shape, at, swap):
    # x and the result are two parts of one array: [tokens, part, heads, dims] and the other orders of those
    g = _gen(sum(shape) + at)
    buf = torch.randn(*shape, generator=g).bfloat16().cuda()
    before = buf.clone()
    parts = [buf.select(at, i) for i in range(shape[at])]
    parts = [t.transpose(0, 1) for t in parts] if swap else parts
    x, out = parts[2], parts[1]                          # in front of x
    f = dsa.dsa_rope_frequencies(32)[0].cuda()
    want = _rope_reference(x.cpu(), f.cpu(), torch.arange(len(x)) + 7, 16, True, 1.0, False)
    assert dsa.dsa_rope(x, f, pos0=7, rot_off=16, out=out).data_ptr() == out.data_ptr()
    _rope_close(out, want, x.cpu(), 1.0)
    back = parts[0]
    dsa.dsa_rope_backward(x, f, pos0=7, rot_off=16, dx=back)
    _rope_close(back, _rope_reference(x.cpu(), f.cpu(), torch.arange(len(x)) + 7, 16, True, 1.0, True), x.cpu(), 1.0)
    keep = torch.ones(shape[at], dtype=torch.bool, device="cuda")
    keep[:2] = False
    assert torch.equal(buf.movedim(at, 0)[keep], before.movedim(at, 0)[keep])
    # parts that have rows in common are refused, before anything is launched
    wide = torch.randn(5, 6, 64, generator=g).bfloat16().cuda()
    for a, b in ((wide[:, :4], wide[:, 1:5]), (wide[:4], wide[1:]), (wide[:, :4, :32], wide[:, 1:5, 16:48])):
        with pytest.raises(dsa.DsaError) as e:
            dsa.dsa_rope(a, f, out=b)
        assert e.value.code == 1                         # DSA_ERR_INVALID_ARG
    assert dsa.dsa_get_device_status() == 0


# ------------------------------------------------------------------------------------------------ together
def _training_step(dsa, s, stream=None):
    """One step of a layer: positions, attention, its backward pass, the objective's gradient, the indexer's."""
    qr = dsa.dsa_rope(s["q"], s["f"], rot_off=512, pos0=s["pos0"], stream=stream)
    cr = dsa.dsa_rope(s["c"].unsqueeze(1), s["f"], rot_off=512, stream=stream).squeeze(1)
    out, lse = dsa.dsa_sparse_mla_attn(qr, cr, s["idx"], SCALE, stream=stream)
    dq, dc = dsa.dsa_sparse_mla_attn_backward(qr, cr, s["idx"], out, lse, s["dout"], SCALE, stream=stream)
    dq = dsa.dsa_rope_backward(dq, s["f"], rot_off=512, pos0=s["pos0"], dx=dq, stream=stream)
    dc = dsa.dsa_rope_backward(dc.unsqueeze(1), s["f"], rot_off=512, stream=stream).squeeze(1)
    dsel = dsa.dsa_indexer_kl_backward(qr, cr, s["idx"], s["sel"], lse, None, SCALE, stream=stream)
    return (dq, dc) + dsa.dsa_indexer_scores_backward(s["q_idx"], s["qs"], s["k_idx"], s["ks"], s["w"], s["idx"], dsel, stream=stream)


def _step_inputs(dsa, seed, T=24, S=400, H=32, k=192):
    q, c, idx, dout = _attention_case(T, S, H, k, "causal", seed)
    qi, qs, ki, ks, w, _, _ = _indexer_case(T, S, 64, 128, k, "causal", True, seed)
    s = dict(q=q, c=c, idx=idx, dout=dout, q_idx=qi, qs=qs, k_idx=ki, ks=ks, w=w, sel=torch.randn(T, k, generator=_gen(seed)))
    s = {n: t.cuda() for n, t in s.items()}
    return dict(s, f=dsa.dsa_rope_frequencies(64)[0].cuda(), pos0=S - T)


def test_training_step(dsa):
    s = _step_inputs(dsa, 21)
    got = _training_step(dsa, s)
    h = {n: t.cpu() for n, t in s.items() if isinstance(t, torch.Tensor)}
    T, S = h["q"].shape[0], h["c"].shape[0]
    q, c = h["q"].double().requires_grad_(), h["c"].double().requires_grad_()

    def turn(x, pos):
        theta = pos.double()[:, None] * h["f"][None]
        cos, sin = theta.cos(), theta.sin()
        a, b = x[..., 512::2], x[..., 513::2]
        if x.dim() == 3:
            cos, sin = cos[:, None], sin[:, None]
        return torch.cat([x[..., :512], torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)], -1)

    qr, cr = turn(q, torch.arange(T) + S - T), turn(c, torch.arange(S))
    out, _, p, _ = _attention(qr, cr, h["idx"])
    out.backward(h["dout"].double())
    # the rotated dims are rounded to bf16 before and after the products: two roundings more
    assert _rel(got[0], q.grad) <= 4 * L2_BF16 and _rel(got[1], c.grad) <= 4 * L2_BF16
    on = h["idx"] >= 0
    target = p.detach().sum(1) / p.shape[1]
    dsel = torch.where(on, torch.softmax(h["sel"].double().masked_fill(~on, -1e300), 1) - target, 0.0)
    qf = (h["q_idx"].float().double() * h["qs"].double()[:, None, None]).requires_grad_()
    kf = (h["k_idx"].float().double() * h["ks"].double()[:, None]).requires_grad_()
    wf = h["w"].double().requires_grad_()
    (_indexer_scores(qf, kf, wf, h["idx"]) * dsel).sum().backward()
    for a, b in zip(got[2:], (qf.grad, kf.grad, wf.grad)):
        assert _rel(a, b) <= 2 * L2_BF16


def test_training_step_on_streams_and_in_graphs(dsa):
    a, b = _step_inputs(dsa, 31), _step_inputs(dsa, 32)
    want_a, want_b = _training_step(dsa, a), _training_step(dsa, b)
    torch.cuda.synchronize()
    # two calls at once on streams of their own
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    ga, gb = _training_step(dsa, a, sa), _training_step(dsa, b, sb)
    torch.cuda.synchronize()
    for x, y in zip(ga + gb, want_a + want_b):
        assert torch.equal(x, y)
    # captured, replayed on new contents of the same buffers, two graphs in turn
    graphs, outs = [], []
    for s in (a, b):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(_training_step(dsa, s))
        graphs.append(graph)
    for n, t in a.items():
        if isinstance(t, torch.Tensor) and n != "f":
            t.copy_(b[n])
    for _ in range(2):
        graphs[0].replay()
        graphs[1].replay()
    torch.cuda.synchronize()
    for x, y in zip(outs[0] + outs[1], want_b + want_b):
        assert torch.equal(x, y)
    assert dsa.dsa_get_device_status() == 0


def test_empty_work(dsa):
    c = torch.randn(30, D).bfloat16().cuda()
    e = lambda *shape, dt=torch.bfloat16: torch.empty(*shape, dtype=dt, device="cuda")
    dq, dc = dsa.dsa_sparse_mla_attn_backward(e(0, 8, D), c, e(0, 128, dt=torch.int32), e(0, 8, DV),
                                              e(0, 8, dt=torch.float32), e(0, 8, DV), SCALE, dc=torch.ones_like(c))
    assert dq.shape == (0, 8, D) and (dc == 0).all()
    k = torch.zeros(30, 128, device="cuda").to(torch.float8_e4m3fn)
    _, dk, dw = dsa.dsa_indexer_scores_backward(e(0, 64, 128, dt=torch.float8_e4m3fn), None, k, None,
                                                e(0, 64, dt=torch.float32), e(0, 128, dt=torch.int32),
                                                e(0, 128, dt=torch.float32), dk=torch.ones(30, 128, device="cuda").bfloat16())
    assert (dk == 0).all() and dw.shape == (0, 64)
