"""The training-side operators on the host (no GPU needed): refusals before anything is launched, workspace sizes, and the
rotary frequencies against their definition."""
import ctypes
import math

import pytest
import torch

P = ctypes.c_void_p
ONE = P(16)            # a dummy aligned non-null address: every call below must fail before touching it
OK, INVALID, SHAPE, ALIGN, WS = 0, 1, 2, 3, 7


@pytest.fixture(scope="module")
def lib():
    import importlib.util
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    spec = importlib.util.spec_from_file_location("dsa_build", os.path.join(root, "sparse_attention_long_05_b200", "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    b.build()
    from sparse_attention_long_05_b200 import _lib
    return _lib._lib


# ------------------------------------------------------------------------------------------- attention backward
ATTN = dict(q=ONE, c=ONE, S=100, idx=ONE, out=ONE, lse=ONE, dout=ONE, T=4, H=8, k=128, scale=1.0, dq=ONE, dc=ONE, ws=ONE,
            ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), INVALID), (dict(S=0), INVALID), (dict(H=0), INVALID), (dict(k=0), INVALID), (dict(dc=None), INVALID),
    (dict(q=None), INVALID), (dict(c=None), INVALID), (dict(idx=None), INVALID), (dict(out=None), INVALID),
    (dict(lse=None), INVALID), (dict(dout=None), INVALID), (dict(dq=None), INVALID),
    (dict(H=129), SHAPE), (dict(k=64), SHAPE), (dict(k=200), SHAPE), (dict(k=2112), SHAPE),
    (dict(q=P(8)), ALIGN), (dict(c=P(24)), ALIGN), (dict(idx=P(4)), ALIGN), (dict(out=P(2)), ALIGN), (dict(dout=P(8)), ALIGN),
    (dict(dq=P(8)), ALIGN), (dict(dc=P(8)), ALIGN), (dict(ws=P(8)), ALIGN),
    (dict(ws=None), WS), (dict(ws_bytes=1 << 10), WS)])
def test_attention_backward_refusals(lib, change, code):
    assert lib.dsa_sparse_mla_attn_backward(*dict(ATTN, **change).values()) == code


def test_attention_backward_workspace(lib):
    size = lib.dsa_sparse_mla_attn_backward_workspace_size
    assert size(0, 100, 8, 128) == size(4, 0, 8, 128) == size(4, 100, 129, 128) == size(4, 100, 8, 100) == 0
    small = size(1, 100, 8, 128)
    assert 0 < small < 1 << 21
    # P, dS and the contributions of every entry fit while a chunk holds all tokens
    n = size(64, 1000, 128, 2048)
    assert n >= 64 * 2048 * (576 * 2 + 4 * 128) + 1000 * 64 * 2
    # longer batches work in chunks of about 4 GiB and keep fp32 sums of every row
    assert size(100000, 32768, 128, 2048) <= (4 << 30) + (1 << 28) + 32768 * 576 * 4
    # one byte less is refused
    assert lib.dsa_sparse_mla_attn_backward(*dict(ATTN, ws_bytes=size(4, 100, 8, 128) - 1).values()) == WS


# ------------------------------------------------------------------------------------------- objective
KL = dict(q=ONE, c=ONE, S=100, idx=ONE, sel=ONE, lse=ONE, dkl=None, T=4, H=8, k=128, scale=1.0, dsel=ONE, ws=ONE,
          ws_bytes=1 << 20, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), INVALID), (dict(S=0), INVALID), (dict(H=0), INVALID), (dict(k=0), INVALID), (dict(q=None), INVALID),
    (dict(c=None), INVALID), (dict(idx=None), INVALID), (dict(sel=None), INVALID), (dict(lse=None), INVALID),
    (dict(dsel=None), INVALID), (dict(H=129), SHAPE), (dict(k=64), SHAPE), (dict(k=2049), SHAPE), (dict(q=P(8)), ALIGN),
    (dict(c=P(8)), ALIGN), (dict(idx=P(8)), ALIGN), (dict(ws=P(8)), ALIGN), (dict(ws=None), WS), (dict(ws_bytes=15), WS),
    (dict(T=0, q=None, c=None, idx=None, sel=None, lse=None, dsel=None, ws=None, ws_bytes=0), OK)])
def test_objective_backward_refusals(lib, change, code):
    assert lib.dsa_indexer_kl_backward(*dict(KL, **change).values()) == code
    assert lib.dsa_indexer_kl_backward_workspace_size(0) == 0 and lib.dsa_indexer_kl_backward_workspace_size(100) >= 400


# ------------------------------------------------------------------------------------------- index scores
INDEX = dict(q=ONE, qs=None, kk=ONE, ks=None, w=ONE, idx=ONE, dsel=ONE, T=4, S=100, H_I=64, d_I=128, k=128, dq=ONE, dk=ONE,
             dw=ONE, ws=ONE, ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), INVALID), (dict(S=0), INVALID), (dict(k=0), INVALID), (dict(q=None), INVALID), (dict(kk=None), INVALID),
    (dict(w=None), INVALID), (dict(idx=None), INVALID), (dict(dsel=None), INVALID), (dict(dq=None), INVALID),
    (dict(dk=None), INVALID), (dict(dw=None), INVALID), (dict(H_I=32), SHAPE), (dict(d_I=64), SHAPE), (dict(k=64), SHAPE),
    (dict(k=2112), SHAPE), (dict(q=P(8)), ALIGN), (dict(kk=P(8)), ALIGN), (dict(idx=P(4)), ALIGN), (dict(dq=P(8)), ALIGN),
    (dict(dk=P(8)), ALIGN), (dict(ws=P(8)), ALIGN), (dict(ws=None), WS), (dict(ws_bytes=100), WS)])
def test_index_scores_backward_refusals(lib, change, code):
    assert lib.dsa_indexer_scores_backward(*dict(INDEX, **change).values()) == code


def test_index_scores_backward_workspace(lib):
    size = lib.dsa_indexer_scores_backward_workspace_size
    assert size(0, 100, 64, 128, 128) == size(4, 100, 64, 64, 128) == size(4, 100, 64, 128, 100) == 0
    assert size(200, 5000, 64, 128, 2048) >= 200 * 2048 * 256 + 5000 * 200 * 2
    assert size(50000, 32768, 64, 128, 2048) <= (4 << 30) + (1 << 27) + 32768 * 128 * 4


def test_workspaces_leave_room_to_align_their_pieces(lib):
    """Every piece of a workspace takes a multiple of 256 bytes, from the workspace's first 256-byte boundary on; a
    workspace may start at any multiple of 16, so up to 240 bytes in front of that boundary come on top."""
    for T, S, H, k in ((1, 8, 1, 128), (4, 100, 8, 192), (300, 70001, 16, 2048)):
        assert lib.dsa_sparse_mla_attn_backward_workspace_size(T, S, H, k) % 256 == 240
        assert lib.dsa_indexer_kl_backward_workspace_size(T) % 256 == 240
        assert lib.dsa_indexer_scores_backward_workspace_size(T, S, 64, 128, k) % 256 == 240
        assert lib.dsa_indexer_scores_backward_workspace_size(T, S, 4, 64, k) % 256 == 240
    need = lib.dsa_indexer_kl_backward_workspace_size(4)
    assert lib.dsa_indexer_kl_backward(*dict(KL, ws=P(32), ws_bytes=need - 1).values()) == WS


# ------------------------------------------------------------------------------------------- rotary positions
ROPE = dict(x=ONE, xt=128, xh=64, out=P(1 << 30), ot=128, oh=64, pos=None, pos0=0, f=ONE, T=4, H=2, D=64, off=0, R=64, inter=1,
            m=1.0, dtype=0, stream=None)


@pytest.mark.parametrize("name", ["dsa_rope", "dsa_rope_backward"])
@pytest.mark.parametrize("change,code", [
    (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(D=0), INVALID), (dict(R=0), INVALID), (dict(R=63), INVALID),
    (dict(off=-1), INVALID), (dict(off=2), INVALID), (dict(R=66), INVALID), (dict(x=None), INVALID), (dict(out=None), INVALID),
    (dict(f=None), INVALID), (dict(dtype=2), INVALID), (dict(xt=-1), INVALID), (dict(pos0=2 ** 31 - 2), INVALID),
    (dict(ot=64), INVALID), (dict(oh=32), INVALID),                     # rows of the result meet
    (dict(out=ONE, ot=256), INVALID),                                  # in place with other strides
    (dict(out=P(16 + 2 * 32)), INVALID),                               # overlapping by half a row
    (dict(x=P(17)), ALIGN), (dict(out=P((1 << 30) + 1)), ALIGN), (dict(f=P(20)), ALIGN), (dict(pos=P(18)), ALIGN),
    (dict(x=P(18), dtype=1), ALIGN), (dict(T=0, x=None, out=None, f=None), OK)])
def test_rope_refusals(lib, name, change, code):
    assert getattr(lib, name)(*dict(ROPE, **change).values()) == code


@pytest.mark.parametrize("change", [
    dict(R=0), dict(R=7), dict(base=1.0), dict(base=math.nan), dict(base=math.inf), dict(factor=0.5), dict(factor=math.nan),
    dict(factor=math.inf, orig=4096), dict(factor=4.0, orig=0), dict(factor=4.0, orig=4096, slow=0.0),
    dict(factor=4.0, orig=4096, fast=1.0, slow=1.0), dict(f=None)])
def test_rope_frequencies_refusals(lib, change):
    out = (ctypes.c_double * 64)()
    a = dict(dict(R=64, base=10000.0, factor=1.0, orig=0, fast=32.0, slow=1.0, f=ctypes.cast(out, P)), **change)
    assert lib.dsa_rope_frequencies(a["R"], a["base"], a["factor"], a["orig"], a["fast"], a["slow"], a["f"], None) == INVALID


def test_rope_frequencies():
    import sparse_attention_long_05_b200 as dsa
    for R, base in ((64, 10000.0), (2, 500000.0), (128, 1e6)):
        f, m = dsa.dsa_rope_frequencies(R, base)
        want = torch.tensor([base ** (-2 * i / R) for i in range(R // 2)], dtype=torch.float64)
        assert m == 1.0 and torch.allclose(f, want, rtol=1e-14, atol=0)
        g, m = dsa.dsa_rope_frequencies(R, base, factor=16.0, orig_len=8192)
        assert m == pytest.approx(0.1 * math.log(16.0) + 1.0, rel=1e-6)
        turns = 8192 * want / (2 * math.pi)
        ratio = g / want
        # fast pairs are kept, slow ones slowed by the factor, none outside; the blend falls with i
        assert ((ratio <= 1 + 1e-12) & (ratio >= 1 / 16 - 1e-12)).all()
        assert (ratio[turns > 32 * 1.5] > 1 - 1e-12).all() or R == 2
        assert (ratio[turns < 1 / 1.5] < 1 / 16 + 1e-12).all()
        assert (ratio[1:] <= ratio[:-1] + 1e-12).all()


@pytest.mark.parametrize("R,base,factor,orig,fast,slow", [
    (64, 1e4, 40.0, 65536, 32.0, 1.0), (64, 1e4, 40.0, 163840, 32.0, 1.0), (16, 1e4, 8.0, 32768, 32.0, 1.0),
    (64, 1e4, 4.0, 1_300_000, 32.0, 1.0), (64, 1e4, 40.0, 4096, 32.0, 1.0), (128, 1e6, 16.0, 8192, 32.0, 1.0),
    (2, 5e5, 16.0, 8192, 32.0, 1.0), (2, 5e5, 16.0, 64, 32.0, 1.0), (64, 1e4, 8.0, 2_000_000_000, 32.0, 1.0),
    (64, 1e4, 8.0, 100, 32.0, 1.0), (64, 1e4, 8.0, 4, 32.0, 1.0), (32, 150000.0, 2.0, 4096, 8.0, 0.5)])
def test_rope_frequencies_blend(R, base, factor, orig, fast, slow):
    """The blend written out pair by pair, also where its ends lie outside the pairs that there are: with orig_len 65536 the
    slowest of 32 pairs still turns 1.39 times and must not be slowed by the whole factor."""
    import sparse_attention_long_05_b200 as dsa
    got, _ = dsa.dsa_rope_frequencies(R, base, factor, orig, fast, slow)
    low = math.floor(R * math.log(orig / (2 * math.pi * fast)) / (2 * math.log(base)))
    high = math.ceil(R * math.log(orig / (2 * math.pi * slow)) / (2 * math.log(base)))
    for i in range(R // 2):
        f = base ** (-2 * i / R)
        r = min(1.0, max(0.0, (i - low) / (high - low)))
        # log, pow and the blend in fp64 on both sides: a few units of 2^-53 each
        assert float(got[i]) == pytest.approx(f * (1 - r + r / factor), rel=1e-13)
        turns = orig * f / (2 * math.pi)
        assert turns <= fast or r == 0.0                          # kept
        assert turns >= slow or r == 1.0                          # slowed by the whole factor
        assert turns <= slow * base ** (2 / R) or r < 1.0         # and no pair a whole index away from those


def test_python_checks_name_the_argument():
    # CPU tensors never reach the library; shapes and types are checked before any pointer is taken
    import sparse_attention_long_05_b200 as dsa
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)
    f = torch.zeros(32, dtype=torch.float64)
    with pytest.raises(ValueError, match="device tensors"):
        dsa.dsa_rope(z(2, 1, 64), f)
    with pytest.raises(ValueError, match="bf16 or fp32"):
        dsa.dsa_rope(z(2, 1, 64, dt=torch.float16), f)
    with pytest.raises(ValueError, match=r"\[T, H, D\]"):
        dsa.dsa_rope(z(2, 64), f)
    with pytest.raises(ValueError, match="device tensors"):
        dsa.dsa_sparse_mla_attn_backward(z(2, 4, 576), z(9, 576), z(2, 128, dt=torch.int32), z(2, 4, 512),
                                         z(2, 4, dt=torch.float32), z(2, 4, 512), 1.0)
    from sparse_attention_long_05_b200 import _lib
    cpu = torch.device("cpu")
    with pytest.raises(ValueError, match="lse is torch.float32 .2, 4."):
        _lib._want("fn", cpu, (("q", z(3), torch.bfloat16, (3,)), ("lse", z(2, 4, dt=torch.float32), torch.float32, (2, 5))))
    with pytest.raises(ValueError, match="idx is torch.int64"):
        _lib._want("fn", cpu, (("idx", z(2, dt=torch.int64), torch.int32, (2,)),))
    with pytest.raises(ValueError, match="contiguous"):
        _lib._want("fn", cpu, (("q", z(4, 4).t(), torch.bfloat16, (4, 4)),))
    assert _lib._want("fn", cpu, (("a", None, torch.int32, (2,)),)) == [None]


def test_integers_beyond_32_bits_are_refused():
    # ctypes would pass their lowest 32 bits on: position 2^32 + 5 as 5, dim 2^32 as 0
    import sparse_attention_long_05_b200 as dsa
    x, f = torch.zeros(2, 1, 64), torch.zeros(32, dtype=torch.float64)
    for call in (dsa.dsa_rope, dsa.dsa_rope_backward):
        for kw in (dict(pos0=2 ** 32 + 5), dict(pos0=2 ** 31), dict(pos0=-2 ** 31 - 1), dict(rot_off=2 ** 32)):
            with pytest.raises(ValueError, match="outside the 32-bit integers"):
                call(x, f, **kw)
    for a, kw in ((2 ** 32 + 64, {}), (64, dict(factor=4.0, orig_len=2 ** 32 + 4096))):
        with pytest.raises(ValueError, match="outside the 32-bit integers"):
            dsa.dsa_rope_frequencies(a, **kw)


def test_rope_backward_takes_one_result():
    import sparse_attention_long_05_b200 as dsa
    x, f = torch.zeros(2, 1, 64), torch.zeros(32, dtype=torch.float64)
    with pytest.raises(ValueError, match="give one of them"):
        dsa.dsa_rope_backward(x, f, dx=torch.zeros(2, 1, 64), out=torch.zeros(2, 1, 64))
