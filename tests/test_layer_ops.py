"""The operators around the recurrence against their 64-bit definitions: the short causal
convolution, the query/key norm with the position rotation, and the selective state space scan,
for prompts and for one token of every beam."""
import ctypes

import pytest
import torch

import layer_ref as ref
import linear_attention_beam_gdn_b200 as ola
import oracle
import workloads as wl
from linear_attention_beam_gdn_b200 import build as olabuild

BF, F = torch.bfloat16, torch.float32
NAN = float("nan")


@pytest.fixture(scope="module")
def L():
    olabuild.build()
    return ola.lib()


def gen(*shape, dtype=F, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed * 7919 + sum((i + 1) * n for i, n in enumerate(shape)))
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def cu(x):
    return None if x is None else x.cuda()


def close(got, want, tol, what):
    got = got.detach().cpu().double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert torch.isfinite(got).all(), f"{what}: non-finite values"
    over = ((got - want).abs() / tol)
    assert float(over.max() if over.numel() else 0.0) <= 1.0, \
        f"{what}: {float(over.max()):.3g} times the bound, off by {float((got - want).abs().max()):.3g}"


def same(a, b, what):
    a, b = a.detach().cpu(), b.detach().cpu()
    assert a.shape == b.shape and torch.equal(a.view(torch.uint8) if a.dtype == BF else a,
                                              b.view(torch.uint8) if b.dtype == BF else b), what


# ----------------------------------------------------------------------------- refusals (CPU)

def _conv_desc(**kw):
    x = dict(R=2, P=5, C=16, W=4, in_dtype=ola.OLA_F32, silu=1)
    x.update(kw)
    return ola.ConvDesc(*[x.pop(n) for n in ("R", "P", "C", "W", "in_dtype", "silu")],
                        *[x.pop(n, 0) for n in ("x_tok", "x_seq", "y_tok", "y_seq")])


A0 = [1 << 20, 2 << 20, 3 << 20, 4 << 20, 5 << 20, 6 << 20, 7 << 20]   # never dereferenced


@pytest.mark.parametrize("kw,code", [
    (dict(R=0), 1), (dict(P=-1), 1), (dict(C=0), 1), (dict(W=1), 2), (dict(W=5), 2),
    (dict(in_dtype=3), 1), (dict(silu=2), 1), (dict(x_tok=15), 1), (dict(y_tok=15), 1),
    (dict(y_seq=79), 1), (dict(x_seq=-1), 1), (dict(x_tok=1 << 62), 1)])
def test_conv_refuses_shapes(L, kw, code):
    assert L.ola_conv(ctypes.byref(_conv_desc(**kw)), *A0, None) == code
    kw = {("P" if n == "P" else n): v for n, v in kw.items()}
    assert L.ola_conv_step(ctypes.byref(_conv_desc(**kw)), 5, *A0[:4], None, *A0[5:], None) == code


def test_conv_refuses_pointers(L):
    d = _conv_desc()
    assert L.ola_conv(None, *A0, None) == 1
    for i in (0, 1, 5):                                  # x, w, y
        a = list(A0)
        a[i] = None
        assert L.ola_conv(ctypes.byref(d), *a, None) == 1, i
    for i, off in ((0, 2), (1, 2), (2, 1), (3, 2), (4, 2), (5, 1), (6, 2)):
        a = list(A0)
        a[i] += off
        assert L.ola_conv(ctypes.byref(d), *a, None) == 1, i
    for i, j in ((5, 0), (5, 1), (5, 3), (6, 0), (5, 6)):  # y or state_out over another tensor
        a = list(A0)
        a[i] = a[j] + 16
        assert L.ola_conv(ctypes.byref(d), *a, None) == 1, (i, j)
    # a step's state: required, in place only without parents and with as many states as beams
    s = [A0[0], A0[1], A0[2], A0[3], None, A0[5], A0[6]]
    d5 = _conv_desc()
    for i in (3, 6):
        a = list(s)
        a[i] = None
        assert L.ola_conv_step(ctypes.byref(d5), 5, *a, None) == 1
    assert L.ola_conv_step(ctypes.byref(d5), 0, *s, None) == 1
    assert L.ola_conv_step(ctypes.byref(d5), 3, *s, None) == 1          # 3 states, 5 beams
    a = list(s)
    a[6] = a[3]
    a[4] = A0[4]
    assert L.ola_conv_step(ctypes.byref(d5), 5, *a, None) == 1          # in place with parents
    a[4] = None
    assert L.ola_conv_step(ctypes.byref(d5), 1, *a, None) == 1          # in place from one state
    assert L.ola_conv_step(ctypes.byref(_conv_desc(P=0)), 5, *s, None) == 1


def _qk_desc(**kw):
    x = dict(N=7, Hq=4, Hk=2, d=64, in_dtype=ola.OLA_BF16, l2=0, rot=32, pair=0, eps=1e-6)
    x.update(kw)
    return ola.QkDesc(*[x.pop(n) for n in ("N", "Hq", "Hk", "d", "in_dtype", "l2", "rot", "pair",
                                           "eps")],
                      *[x.pop(n, 0) for n in ("q_tok", "k_tok", "qo_tok", "ko_tok")])


@pytest.mark.parametrize("kw,code", [
    (dict(N=-1), 1), (dict(Hq=-1), 1), (dict(d=0), 1), (dict(d=12), 2), (dict(d=520), 2),
    (dict(in_dtype=2), 1), (dict(l2=3), 1), (dict(pair=2), 1), (dict(rot=8), 2),
    (dict(rot=80), 2), (dict(rot=-16), 2), (dict(eps=-1.0), 1), (dict(eps=NAN), 1),
    (dict(q_tok=255), 1), (dict(q_tok=257), 1), (dict(ko_tok=129), 1)])
def test_qk_norm_refuses_shapes(L, kw, code):
    assert L.ola_qk_norm(ctypes.byref(_qk_desc(**kw)), *A0, 8 << 20, None) == code


def test_qk_norm_refuses_pointers(L):
    a0 = A0 + [8 << 20]                       # q, k, wq, wk, positions, inv_freq, q_out, k_out
    d = _qk_desc()
    assert L.ola_qk_norm(None, *a0, None) == 1
    for i in (0, 1, 4, 5, 6, 7):
        a = list(a0)
        a[i] = None
        assert L.ola_qk_norm(ctypes.byref(d), *a, None) == 1, i
    for i, off in ((0, 8), (1, 8), (2, 2), (3, 2), (4, 2), (5, 2), (6, 8), (7, 8)):
        a = list(a0)
        a[i] += off
        assert L.ola_qk_norm(ctypes.byref(d), *a, None) == 1, i
    for i, j, off in ((6, 0, 16), (6, 1, 0), (7, 0, 0), (7, 6, 0), (7, 1, 32)):
        a = list(a0)
        a[i] = a[j] + off
        assert L.ola_qk_norm(ctypes.byref(d), *a, None) == 1, (i, j)
    assert L.ola_qk_norm(ctypes.byref(_qk_desc(N=0)), *a0, None) == 0   # nothing to do
    assert L.ola_qk_norm(ctypes.byref(_qk_desc(Hq=0, Hk=0)), *a0, None) == 0


def _scan_desc(**kw):
    x = dict(R=2, P=5, H=4, G=2, d_k=16, d_v=32, in_dtype=ola.OLA_F32, softplus=1)
    x.update(kw)
    return ola.ScanDesc(*[x.pop(n) for n in ("R", "P", "H", "G", "d_k", "d_v", "in_dtype",
                                             "softplus")],
                        *[x.pop(n, 0) for n in ("v_tok", "v_seq", "k_tok", "k_seq", "q_tok",
                                                "q_seq", "z_tok", "z_seq", "y_tok", "y_seq")])


S0 = [(i + 1) << 20 for i in range(12)]     # v dt A k q D dt_bias z S_in lens|parent y S_out


@pytest.mark.parametrize("kw,code", [
    (dict(R=0), 1), (dict(P=-1), 1), (dict(H=0), 1), (dict(G=3), 1), (dict(G=0), 1),
    (dict(d_k=48), 2), (dict(d_v=512), 2), (dict(in_dtype=2), 1), (dict(softplus=2), 1),
    (dict(R=1 << 20, H=1 << 10, G=1), 2), (dict(v_tok=127), 1), (dict(k_tok=31), 1),
    (dict(y_tok=127), 1), (dict(y_seq=1), 1)])
def test_scan_refuses_shapes(L, kw, code):
    d = _scan_desc(**kw)
    assert L.ola_scan(ctypes.byref(d), *S0, None, 0, None) == code
    assert L.ola_scan_step(ctypes.byref(d), 5, *S0, None) == code
    if not any(n.endswith(("tok", "seq")) for n in kw):
        assert L.ola_scan_workspace_bytes(ctypes.byref(d), ctypes.byref(ctypes.c_uint64())) == code


def test_scan_refuses_pointers(L):
    d = _scan_desc()
    assert L.ola_scan(None, *S0, None, 0, None) == 1
    assert L.ola_scan_workspace_bytes(ctypes.byref(d), None) == 1
    for i in (0, 1, 2, 3, 4, 10):
        a = list(S0)
        a[i] = None
        assert L.ola_scan(ctypes.byref(d), *a, None, 0, None) == 1, i
        assert L.ola_scan_step(ctypes.byref(d), 5, *a, None) == 1, i
    for i in range(12):
        a = list(S0)
        a[i] += 2
        assert L.ola_scan(ctypes.byref(d), *a, None, 0, None) == 1, i
        assert L.ola_scan_step(ctypes.byref(d), 5, *a, None) == 1, i
    for i, j in ((10, 0), (10, 3), (10, 1), (10, 8), (11, 0), (11, 10)):
        a = list(S0)
        a[i] = a[j] + 16
        assert L.ola_scan(ctypes.byref(d), *a, None, 0, None) == 1, (i, j)
        a[9] = None
        assert L.ola_scan_step(ctypes.byref(d), 5, *a, None) == 1, (i, j)
    a = list(S0)
    a[11] = a[8]                                        # in place with parents
    assert L.ola_scan_step(ctypes.byref(d), 5, *a, None) == 1
    for i in (8, 11):
        a = list(S0)
        a[i] += 4                                       # a step's states are 16-byte aligned
        assert L.ola_scan_step(ctypes.byref(d), 5, *a, None) == 1
        a[i] = None
        assert L.ola_scan_step(ctypes.byref(d), 5, *a, None) == 1
    # a long prompt of one sequence needs its scratch
    d = _scan_desc(R=1, P=4096, H=1, G=1)
    n = ola.ola_scan_workspace_bytes(d)
    assert n > 0
    far = [(i + 1) << 26 for i in range(12)]
    assert L.ola_scan(ctypes.byref(d), *far, None, n, None) == 1
    assert L.ola_scan(ctypes.byref(d), *far, 13 << 26, n - 1, None) == 1
    assert L.ola_scan(ctypes.byref(d), *far, (13 << 26) + 8, n, None) == 1
    assert L.ola_scan(ctypes.byref(d), *far, far[0], n, None) == 1


def test_refuses_lengths_past_the_limit(L):
    """A sequence of more than 2^30 tokens (or that many beams) is unsupported, not wrapped."""
    n = (1 << 30) + 1
    far = [(i + 1) << 50 for i in range(12)]
    c = _conv_desc(R=1, P=n, C=8)
    assert L.ola_conv(ctypes.byref(c), *far[:7], None) == 2
    assert L.ola_conv_step(ctypes.byref(c), 1, *far[:4], None, *far[5:7], None) == 2
    d = _scan_desc(R=1, P=n, H=1, G=1, d_k=16, d_v=16)
    assert L.ola_scan(ctypes.byref(d), *far, None, 0, None) == 2
    assert L.ola_scan_step(ctypes.byref(d), 1, *far, None) == 2
    assert L.ola_scan_workspace_bytes(ctypes.byref(d), ctypes.byref(ctypes.c_uint64())) == 2


def test_wrappers_refuse_tensors(L):
    x, w = torch.zeros(1, 4, 8), torch.zeros(8, 4)
    with pytest.raises(ValueError):
        ola.conv(x, w)                                   # not on a CUDA device
    with pytest.raises(TypeError):
        ola.conv([1.0], w)
    with pytest.raises(ValueError):
        ola.qk_norm(torch.zeros(1, 2, 1, 64), torch.zeros(1, 2, 1, 64))
    with pytest.raises(ValueError):
        ola.scan(torch.zeros(1, 2, 1, 64), None, None, None, None)


# ----------------------------------------------------------------------------- convolution

CONV = [  # dtype, R, P, C, W, bias, state, lens, silu
    (F, 1, 1, 8, 4, False, False, None, True),
    (F, 2, 2, 12, 3, True, True, None, True),
    (F, 3, 37, 33, 4, True, True, [37, 0, 2], False),
    (F, 2, 131, 520, 2, False, True, [1, 500], True),
    (BF, 1, 1, 8, 2, True, False, None, True),
    (BF, 1, 3, 1001, 4, False, True, None, False),
    (BF, 4, 70, 264, 4, True, True, [70, -3, 1, 69], True),
    (BF, 2, 200, 72, 3, True, False, None, True),
    (BF, 5, 33, 2048, 4, False, True, [33, 32, 31, 3, 0], True),
]


def _conv_case(dtype, R, P, C, W, bias, state, lens):
    x, w = gen(R, P, C, dtype=dtype), gen(C, W, seed=1)
    b = gen(C, seed=2) if bias else None
    st = gen(R, W - 1, C, dtype=dtype, seed=3) if state else None
    ln = torch.tensor(lens, dtype=torch.int32) if lens is not None else None
    return x, w, b, st, ln


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,R,P,C,W,bias,state,lens,act", CONV)
def test_conv_against_definition(dtype, R, P, C, W, bias, state, lens, act):
    x, w, b, st, ln = _conv_case(dtype, R, P, C, W, bias, state, lens)
    out0 = torch.full((R, P, C), 7.0, dtype=dtype)
    y64, s64, tol = ref.conv(x, w, b, st, ln, act, out0)
    xg = x.clone()
    if lens is not None:                                 # padding holds anything
        for r, n in enumerate(lens):
            xg[r, max(0, min(P, n)):] = NAN
    y, s = ola.conv(xg.cuda(), w.cuda(), cu(b), state=cu(st), lens=cu(ln), silu=act,
                    out=out0.cuda())
    close(y, y64, tol, "y")
    assert torch.equal(s.cpu().double(), s64), "state"   # moved, not computed
    assert ola.layer_status() == ola.OLA_OK


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,C,off,wide", [(BF, 64, 0, 192), (BF, 64, 3, 70), (F, 20, 4, 40),
                                              (F, 7, 1, 9)])
def test_conv_column_slices(dtype, C, off, wide):
    """x and y are column slices of one buffer; the other columns and rows stay as they were."""
    R, P, W = 2, 45, 4
    big = gen(R, P, 2 * wide, dtype=dtype)
    w = gen(C, W, seed=1)
    g = big.cuda()
    x, out = g[:, :, off:off + C], g[:, :, wide + off:wide + off + C]
    y64, s64, tol = ref.conv(big[:, :, off:off + C].contiguous(), w, None, None, None, True,
                             torch.zeros(R, P, C, dtype=dtype))
    _, s = ola.conv(x, w.cuda(), out=out)
    close(out, y64, tol, "y")
    assert torch.equal(s.cpu().double(), s64)
    rest = g.cpu()
    rest[:, :, wide + off:wide + off + C] = big[:, :, wide + off:wide + off + C]
    same(rest, big, "other columns")
    with pytest.raises(ola.OlaError):
        ola.conv(x, w.cuda(), out=x)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F])
def test_conv_pieces_and_steps_equal_the_whole(dtype):
    """A prompt in one call, in pieces that carry the state in place, and token by token: bit for bit."""
    R, P, C, W = 3, 50, 136, 4
    x, w, b, st, _ = _conv_case(dtype, R, P, C, W, True, True, None)
    x, w, b, st = x.cuda(), w.cuda(), b.cuda(), st.cuda()
    y, s = ola.conv(x, w, b, state=st)
    cur, parts = st.clone(), []
    for p0, p1 in ((0, 1), (1, 3), (3, 33), (33, 33), (33, 50)):
        yp, cur2 = ola.conv(x[:, p0:p1].contiguous(), w, b, state=cur, state_out=cur)
        assert cur2 is cur
        parts.append(yp)
    same(torch.cat(parts, 1), y, "pieces")
    same(cur, s, "state of the pieces")
    cur = st[:, None].clone()
    for p in range(P):
        yp, _ = ola.conv_step(x[:, p:p + 1], w, b, state=cur, state_out=cur)
        same(yp[:, 0], y[:, p], f"token {p}")
    same(cur[:, 0], s, "state of the steps")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,R,B,Bp,C,W", [(BF, 1, 1, 1, 64, 4), (BF, 3, 37, 37, 264, 4),
                                              (F, 2, 5, 1, 33, 3), (BF, 2, 16, 40, 1001, 2),
                                              (F, 4, 64, 8, 128, 4)])
@pytest.mark.parametrize("with_parents", [True, False])
def test_conv_step_beams(dtype, R, B, Bp, C, W, with_parents):
    if not with_parents and Bp not in (1, B):
        Bp = B
    x, w, b = gen(R, B, C, dtype=dtype), gen(C, W, seed=1), gen(C, seed=2)
    st = gen(R, Bp, W - 1, C, dtype=dtype, seed=3)
    par = (torch.arange(R * B).reshape(R, B) * 7 % 3 % Bp).int() if with_parents else None
    pick = par.long() if with_parents else (torch.arange(B) % Bp).expand(R, B)
    chosen = st[torch.arange(R)[:, None], pick]                       # [R, B, W-1, C]
    y64, s64, tol = ref.conv(x.reshape(R * B, 1, C), w, b, chosen.reshape(R * B, W - 1, C), None,
                             True, torch.zeros(R * B, 1, C, dtype=dtype))
    y, s = ola.conv_step(x.cuda(), w.cuda(), b.cuda(), state=st.cuda(), parent_idx=cu(par))
    close(y.reshape(R * B, 1, C), y64, tol, "y")
    assert torch.equal(s.cpu().double().reshape(R * B, W - 1, C), s64)


@pytest.mark.gpu
def test_bad_parents_are_recorded_and_clamped():
    R, B, C, W = 1, 4, 16, 4
    x, w, st = gen(R, B, C).cuda(), gen(C, W, seed=1).cuda(), gen(R, B, W - 1, C, seed=3).cuda()
    good = torch.tensor([[0, 1, 0, 0]], dtype=torch.int32).cuda()
    bad = torch.tensor([[0, 1, 4, -1]], dtype=torch.int32).cuda()
    assert ola.layer_status() == ola.OLA_OK
    y0, s0 = ola.conv_step(x, w, state=st, parent_idx=good)
    y1, s1 = ola.conv_step(x, w, state=st, parent_idx=bad)
    assert ola.layer_status() == ola.OLA_ERR_BAD_PARENT
    assert ola.layer_status() == ola.OLA_OK
    same(y0, y1, "y")
    same(s0, s1, "state")
    v, k = gen(R, B, 2, 16, seed=4).cuda(), gen(R, B, 2, 32, seed=5).cuda()
    dt, A = gen(R, B, 2, seed=6).cuda(), -torch.ones(2).cuda()
    st = gen(R, B, 2, 16, 32, seed=7).cuda()
    y0, s0 = ola.scan_step(v, dt, A, k, k, state=st, parent_idx=good)
    y1, s1 = ola.scan_step(v, dt, A, k, k, state=st, parent_idx=bad)
    assert ola.layer_status() == ola.OLA_ERR_BAD_PARENT
    same(y0, y1, "y")
    same(s0, s1, "state")


@pytest.mark.gpu
def test_conv_far_offsets():
    """Rows more than 2^32 elements apart."""
    C, W, P = 64, 4, 9
    tok = (1 << 30) + 64
    big = torch.empty((1, P, tok), device="cuda", dtype=BF)
    x = gen(1, P, C, dtype=BF)
    big[:, :, :C] = x.cuda()
    w = gen(C, W, seed=1)
    y64, s64, tol = ref.conv(x, w, None, None, None, True, torch.zeros(1, P, C, dtype=BF))
    y, s = ola.conv(big[:, :, :C], w.cuda(), out=big[:, :, 128:128 + C])
    close(y, y64, tol, "y")
    assert torch.equal(s.cpu().double(), s64)


# ----------------------------------------------------------------------------- query/key norm

QK = [  # dtype, R, P, Hq, Hk, d, rot, pair, l2, weights
    (BF, 1, 1, 1, 1, 8, 0, False, False, False),
    (BF, 2, 5, 4, 2, 64, 64, False, False, True),
    (BF, 1, 7, 16, 16, 128, 0, False, True, False),
    (BF, 3, 3, 5, 1, 80, 48, False, False, True),
    (BF, 1, 9, 2, 3, 256, 64, True, False, True),
    (BF, 1, 4, 3, 1, 512, 512, False, True, True),
    (BF, 2, 2, 7, 0, 24, 16, True, False, False),
    (BF, 2, 2, 0, 7, 104, 96, False, False, True),
    (F, 1, 1, 1, 1, 16, 16, True, False, False),
    (F, 2, 6, 4, 4, 64, 32, False, True, False),
    (F, 1, 5, 3, 2, 128, 128, False, False, True),
    (F, 1, 3, 2, 1, 512, 256, True, False, True),
    (F, 1, 3, 2, 1, 264, 256, False, False, True),
    (F, 1, 2, 2, 5, 40, 32, False, True, True),
]


def _qk_case(dtype, R, P, Hq, Hk, d, rot, weights):
    q, k = gen(R, P, Hq, d, dtype=dtype, seed=1), gen(R, P, Hk, d, dtype=dtype, seed=2, scale=3.0)
    wq, wk = (gen(d, seed=3), gen(d, seed=4)) if weights else (None, None)
    pos = inv = None
    if rot:
        g = torch.Generator().manual_seed(5)
        pos = torch.randint(-10, 1 << 20, (R, P), generator=g, dtype=torch.int32)
        pos.view(-1)[0] = (1 << 31) - 1
        inv = (1e4 ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / rot)).float()
    return q, k, wq, wk, pos, inv


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,R,P,Hq,Hk,d,rot,pair,l2,weights", QK)
def test_qk_norm_against_definition(dtype, R, P, Hq, Hk, d, rot, pair, l2, weights):
    q, k, wq, wk, pos, inv = _qk_case(dtype, R, P, Hq, Hk, d, rot, weights)
    eps = 1e-6
    q64, qt = ref.qk_norm(q, wq, eps, l2, pos, inv, pair)
    k64, kt = ref.qk_norm(k, wk, eps, l2, pos, inv, pair)
    args = dict(wq=cu(wq), wk=cu(wk), eps=eps, l2=l2, positions=cu(pos), inv_freq=cu(inv),
                pair=pair)
    qo, ko = ola.qk_norm(q.cuda(), k.cuda(), **args)
    close(qo, q64, qt, "q")
    close(ko, k64, kt, "k")
    # in place, and as column slices of one projection
    qi, ki = q.cuda(), k.cuda()
    ola.qk_norm(qi, ki, **args, q_out=qi, k_out=ki)
    same(qi, qo, "q in place")
    same(ki, ko, "k in place")
    wide = torch.full((R, P, (Hq + Hk + 1) * d), 5.0, device="cuda", dtype=dtype)
    qs = wide[:, :, :Hq * d].unflatten(2, (Hq, d))
    ks = wide[:, :, Hq * d:(Hq + Hk) * d].unflatten(2, (Hk, d))
    qs.copy_(q)
    ks.copy_(k)
    ola.qk_norm(qs, ks, **args, q_out=qs, k_out=ks)
    same(qs.contiguous(), qo, "q slice")
    same(ks.contiguous(), ko, "k slice")
    assert bool((wide[:, :, (Hq + Hk) * d:] == 5.0).all())


@pytest.mark.gpu
def test_qk_norm_special_values():
    """A zero head stays zero (eps > 0); a NaN or infinity stays within its head."""
    q = gen(1, 2, 3, 64, dtype=BF)
    q[0, 0, 1] = 0
    q[0, 1, 2, 5] = float("inf")
    q[0, 1, 0, 7] = NAN
    k = gen(1, 2, 1, 64, dtype=BF, seed=1)
    qo, ko = ola.qk_norm(q.cuda(), k.cuda())
    assert bool((qo[0, 0, 1] == 0).all())
    fine = torch.isfinite(qo).all(-1).cpu()
    assert fine.tolist() == [[[True, True, True], [False, True, False]]]
    assert bool(torch.isfinite(ko).all())
    e = torch.zeros(0, 1, device="cuda", dtype=torch.int32)
    z = torch.zeros(0, 1, 2, 64, device="cuda", dtype=BF)
    qo, ko = ola.qk_norm(z, z, positions=e, inv_freq=torch.ones(8, device="cuda"))
    assert qo.shape == z.shape


@pytest.mark.gpu
def test_qk_norm_many_tokens_equal_few():
    """The split of a token's heads over warps hangs on the number of tokens; the results do not."""
    q, k = gen(1, 6000, 6, 128, dtype=BF).cuda(), gen(1, 6000, 2, 128, dtype=BF, seed=1).cuda()
    pos = torch.arange(6000, dtype=torch.int32, device="cuda")[None]
    inv = (1e4 ** (-torch.arange(64, dtype=torch.float64) / 64)).float().cuda()
    qo, ko = ola.qk_norm(q, k, positions=pos, inv_freq=inv)
    for p in (0, 1, 2999, 5999):
        qp, kp = ola.qk_norm(q[:, p:p + 1], k[:, p:p + 1], positions=pos[:, p:p + 1].contiguous(),
                             inv_freq=inv)
        same(qp, qo[:, p:p + 1], "q")
        same(kp, ko[:, p:p + 1], "k")


# ----------------------------------------------------------------------------- scan

def _scan_case(dtype, R, P, H, G, dk, dv, z=False, D=False, bias=True, state=False, lens=None,
               softplus=True, seed=0):
    s = seed * 100
    c = dict(v=gen(R, P, H, dv, dtype=dtype, seed=s + 1), dt=gen(R, P, H, seed=s + 2),
             A=-torch.rand(H, generator=torch.Generator().manual_seed(s)) * 8 - 0.05,
             k=gen(R, P, G, dk, dtype=dtype, seed=s + 3, scale=dk ** -0.5),
             q=gen(R, P, G, dk, dtype=dtype, seed=s + 4))
    if not softplus:
        c["dt"] = c["dt"].abs() * 0.2
    o = dict(D=gen(H, seed=s + 5) if D else None,
             dt_bias=gen(H, seed=s + 6) - 3.0 if bias else None,
             z=gen(R, P, H, dv, dtype=dtype, seed=s + 7) if z else None,
             S_in=gen(R, H, dv, dk, seed=s + 8) if state else None,
             lens=torch.tensor(lens, dtype=torch.int32) if lens is not None else None)
    if not softplus and bias:
        o["dt_bias"] = o["dt_bias"].abs() * 0.01
    return c, o


def _chunked(dtype, dk):
    return dtype == BF and dk <= 128


SCAN = [  # dtype, R, P, H, G, dk, dv, options
    (F, 1, 1, 1, 1, 16, 16, {}),
    (F, 2, 33, 4, 2, 32, 16, dict(z=True, D=True, state=True, lens=[33, 5])),
    (F, 1, 70, 2, 1, 64, 32, dict(D=True)),
    (F, 2, 40, 3, 3, 128, 64, dict(z=True, lens=[0, 40], state=True)),
    (F, 1, 37, 2, 2, 256, 128, dict(state=True)),
    (F, 1, 35, 1, 1, 16, 256, dict(softplus=False)),
    (F, 1, 600, 1, 1, 64, 64, dict(state=True, D=True)),            # pieces
    (F, 2, 500, 2, 1, 16, 32, dict(lens=[130, 499], z=True)),       # pieces, one ends early
    (BF, 1, 1, 2, 1, 128, 64, dict(state=True)),
    (BF, 1, 128, 2, 2, 128, 128, {}),
    (BF, 2, 129, 4, 1, 128, 64, dict(z=True, D=True)),
    (BF, 3, 300, 2, 2, 64, 64, dict(lens=[300, 128, 0], state=True, z=True, D=True)),
    (BF, 1, 260, 3, 1, 64, 128, dict(softplus=False)),
    (BF, 2, 140, 2, 2, 32, 32, dict(D=True, lens=[127, 140])),
    (BF, 1, 200, 2, 1, 16, 16, dict(z=True, state=True)),
    (BF, 1, 150, 1, 1, 128, 256, dict(state=True)),
    (BF, 1, 90, 2, 1, 256, 64, dict(z=True, state=True)),
    (BF, 1, 1500, 1, 1, 128, 64, dict(state=True, D=True)),         # pieces
    (BF, 2, 1000, 2, 1, 64, 64, dict(lens=[1000, 385], state=True)),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,R,P,H,G,dk,dv,opt", SCAN)
def test_scan_against_definition(dtype, R, P, H, G, dk, dv, opt):
    c, o = _scan_case(dtype, R, P, H, G, dk, dv, **opt)
    sp = opt.get("softplus", True)
    out0 = torch.full((R, P, H, dv), 3.0, dtype=dtype)
    y64, S64, ty, tS = ref.scan(**c, D=o["D"], dt_bias=o["dt_bias"], z=o["z"], S_in=o["S_in"],
                                lens=o["lens"], use_softplus=sp, out0=out0,
                                chunked=_chunked(dtype, dk))
    cg = {n: t.clone() for n, t in c.items()}
    zg = None if o["z"] is None else o["z"].clone()
    if o["lens"] is not None:
        for r, n in enumerate(opt["lens"]):
            for t in (cg["v"], cg["dt"], cg["k"], cg["q"]) + (() if zg is None else (zg,)):
                t[r, n:] = NAN
    cg = {n: t.cuda() for n, t in cg.items()}
    kw = dict(D=cu(o["D"]), dt_bias=cu(o["dt_bias"]), z=cu(zg), lens=cu(o["lens"]), softplus=sp)
    S_in = cu(o["S_in"])
    y, S = ola.scan(**cg, **kw, S_in=S_in, out=out0.cuda())
    assert ola.layer_status() == ola.OLA_OK
    close(y, y64, ty, "y")
    close(S, S64, tS, "state")
    if S_in is not None:                                # the state replaced in place
        y2, S2 = ola.scan(**cg, **kw, S_in=S_in, S_out=S_in, out=out0.cuda())
        same(y2, y, "y, state in place")
        same(S2, S, "state in place")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F])
def test_scan_decays_of_every_size(dtype):
    """Resets (a decay that underflows), no decay at all, and both side by side."""
    R, P, H, dk, dv = 1, 300, 3, 64, 64
    c, o = _scan_case(dtype, R, P, H, 1, dk, dv, bias=False, softplus=False, state=True)
    c["dt"][:] = 0.05
    c["dt"][0, 40::50] = 60.0                            # with A = -8: exp(-480)
    c["dt"][0, 100:110] = 0.0                            # nothing decays, nothing is added
    c["A"] = torch.tensor([-8.0, -1e-4, 0.0])
    out0 = torch.zeros(R, P, H, dv, dtype=dtype)
    y64, S64, ty, tS = ref.scan(**c, D=None, dt_bias=None, z=None, S_in=o["S_in"], lens=None,
                                use_softplus=False, out0=out0, chunked=_chunked(dtype, dk))
    y, S = ola.scan(**{n: t.cuda() for n, t in c.items()}, S_in=cu(o["S_in"]), softplus=False)
    close(y, y64, ty, "y")
    close(S, S64, tS, "state")


@pytest.mark.gpu
@pytest.mark.parametrize("dk,z", [(64, False), (64, True), (128, False), (128, True)])
def test_scan_many_chunks_in_one_piece(dk, z):
    """So many heads that no sequence is cut: every stage of the chunk pipeline is used again and
    again, by heads that end at different chunks."""
    R, P, H, dv = 2, 900, 40, 32
    lens = [900, 641]
    c, o = _scan_case(BF, R, P, H, 1, dk, dv, z=z, D=True, state=True, lens=lens, seed=3)
    out0 = torch.full((R, P, H, dv), 3.0, dtype=BF)
    y64, S64, ty, tS = ref.scan(**c, D=o["D"], dt_bias=o["dt_bias"], z=o["z"], S_in=o["S_in"],
                                lens=o["lens"], use_softplus=True, out0=out0, chunked=True)
    cg = {n: t.cuda() for n, t in c.items()}
    first = None
    for _ in range(3):
        y, S = ola.scan(**cg, D=cu(o["D"]), dt_bias=cu(o["dt_bias"]), z=cu(o["z"]),
                        S_in=cu(o["S_in"]), lens=cu(o["lens"]), out=out0.cuda())
        assert ola.layer_status() == ola.OLA_OK
        if first is None:
            close(y, y64, ty, "y")
            close(S, S64, tS, "state")
            first = y, S
        same(y, first[0], "y")
        same(S, first[1], "state")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,H,dk,z,lens", [
    (BF, 2, 128, True, None), (BF, 2, 64, False, [300, 270]), (BF, 2, 32, True, [300, 270]),
    (BF, 40, 16, False, None), (BF, 40, 128, True, [300, 270]), (F, 2, 32, True, None)])
def test_scan_values_that_are_not_finite_stay_causal(dtype, H, dk, z, lens):
    """An infinity or NaN in v reaches its own column, from its own token on, and nothing else."""
    R, P, dv = 2, 300, 64
    c, o = _scan_case(dtype, R, P, H, 1, dk, dv, z=z, D=True, state=True, lens=lens, seed=4)
    c["v"][:, 5::7] = -0.0                               # an ordinary value, also beside the others
    bad = [(0, 10, 0, 63, NAN), (0, 140, 1, 5, float("inf")), (0, 200, 1, 5, -float("inf")),
           (1, 127, 0, 0, -float("inf")), (1, 128, 0, 1, NAN), (1, 255, 1, 33, float("inf")),
           (1, 269, 1, 34, NAN), (1, 160, 1, 31, NAN)]
    dirty = c["v"].clone()
    hit = torch.zeros(R, P, H, dv, dtype=torch.bool)
    for r, p, h, e, x in bad:
        c["v"][r, p, h, e], dirty[r, p, h, e] = 0.0, x
        hit[r, p:P if lens is None else lens[r], h, e] = True
    out0 = torch.full((R, P, H, dv), 3.0, dtype=dtype)
    y64, S64, ty, tS = ref.scan(**c, D=o["D"], dt_bias=o["dt_bias"], z=o["z"], S_in=o["S_in"],
                                lens=o["lens"], use_softplus=True, out0=out0,
                                chunked=_chunked(dtype, dk))
    kw = {n: t.cuda() for n, t in c.items() if n != "v"}
    rows = hit.any(1)                                     # [R, H, dv]
    for in_place in (False, True):
        S_in = cu(o["S_in"])
        y, S = ola.scan(dirty.cuda(), **kw, D=cu(o["D"]), dt_bias=cu(o["dt_bias"]), z=cu(o["z"]),
                        S_in=S_in, S_out=S_in if in_place else None, lens=cu(o["lens"]),
                        out=out0.cuda())
        assert ola.layer_status() == ola.OLA_OK
        y, S = y.cpu(), S.cpu()
        assert not torch.isfinite(y[hit]).any()
        close(y.masked_fill(hit, 0.0), y64.masked_fill(hit, 0.0), ty, "y elsewhere")
        assert not torch.isfinite(S[rows]).any()
        close(S.masked_fill(rows[..., None], 0.0), S64.masked_fill(rows[..., None], 0.0), tS,
              "state elsewhere")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,off", [(BF, 0), (BF, 8), (BF, 3), (F, 4), (F, 1)])
def test_scan_column_slices(dtype, off):
    """v, k, q, z as column slices of one projection, y into another buffer's columns."""
    R, P, H, G, dk, dv = 2, 150, 2, 1, 64, 64
    c, o = _scan_case(dtype, R, P, H, G, dk, dv, z=True)
    kw = dict(dt=c["dt"].cuda(), A=c["A"].cuda())
    want_y, want_S = ola.scan(c["v"].cuda(), kw["dt"], kw["A"], c["k"].cuda(), c["q"].cuda(),
                              z=o["z"].cuda())
    wide = torch.zeros(R, P, off + 2 * H * dv + 2 * G * dk + 8, device="cuda", dtype=dtype)
    parts, at = [], off
    for t in (c["v"], o["z"], c["k"], c["q"]):
        n = t.shape[2] * t.shape[3]
        s = wide[:, :, at:at + n].unflatten(2, t.shape[2:])
        s.copy_(t)
        parts.append(s)
        at += n
    out = torch.full((R, P, H * dv + 16), 9.0, device="cuda", dtype=dtype)
    y = out[:, :, off:off + H * dv].unflatten(2, (H, dv))
    _, S = ola.scan(parts[0], kw["dt"], kw["A"], parts[2], parts[3], z=parts[1], out=y)
    tol = 1e-6 if dtype == F else 2e-2                    # another alignment, another kernel
    assert float((y.float() - want_y.float()).abs().max()) <= tol * float(want_y.abs().max())
    assert float((S - want_S).abs().max()) <= 1e-5 * float(want_S.abs().max())
    left = out.clone()
    left[:, :, off:off + H * dv] = 9.0
    assert bool((left == 9.0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,R,B,Bp,H,G,dk,dv,opt", [
    (BF, 1, 1, 1, 1, 1, 128, 128, {}), (BF, 2, 5, 5, 4, 2, 64, 64, dict(z=True, D=True)),
    (F, 2, 3, 1, 2, 1, 16, 16, dict(D=True)), (F, 1, 7, 9, 3, 3, 32, 64, dict(z=True)),
    (BF, 2, 4, 6, 2, 1, 256, 32, dict(softplus=False)), (F, 1, 2, 2, 2, 2, 128, 256, {})])
@pytest.mark.parametrize("with_parents", [True, False])
def test_scan_step_beams(dtype, R, B, Bp, H, G, dk, dv, opt, with_parents):
    if not with_parents and Bp not in (1, B):
        Bp = B
    c, o = _scan_case(dtype, R, B, H, G, dk, dv, **opt)
    sp = opt.get("softplus", True)
    st = gen(R, Bp, H, dv, dk, seed=9)
    par = (torch.arange(R * B).reshape(R, B) * 5 % Bp).int() if with_parents else None
    pick = par.long() if with_parents else (torch.arange(B) % Bp).expand(R, B)
    chosen = st[torch.arange(R)[:, None], pick].reshape(R * B, H, dv, dk)
    one = {n: (t if n == "A" else t.reshape((R * B, 1) + t.shape[2:])) for n, t in c.items()}
    z1 = None if o["z"] is None else o["z"].reshape(R * B, 1, H, dv)
    y64, S64, ty, tS = ref.scan(**one, D=o["D"], dt_bias=o["dt_bias"], z=z1, S_in=chosen, lens=None,
                                use_softplus=sp, out0=torch.zeros(R * B, 1, H, dv, dtype=dtype))
    kw = dict(D=cu(o["D"]), dt_bias=cu(o["dt_bias"]), z=cu(o["z"]), softplus=sp)
    cg = {n: t.cuda() for n, t in c.items()}
    y, S = ola.scan_step(**cg, **kw, state=st.cuda(), parent_idx=cu(par))
    close(y.reshape(R * B, 1, H, dv), y64, ty, "y")
    close(S.reshape(R * B, H, dv, dk), S64, tS, "state")
    if not with_parents and Bp == B:
        cur = st.cuda()
        y2, S2 = ola.scan_step(**cg, **kw, state=cur, state_out=cur)
        same(y2, y, "y in place")
        same(S2, S, "state in place")


@pytest.mark.gpu
def test_empty_prompt_keeps_the_states():
    S_in = gen(2, 3, 16, 64, seed=1).cuda()
    e = lambda *s, t=BF: torch.zeros(s, device="cuda", dtype=t)  # noqa: E731
    y, S = ola.scan(e(2, 0, 3, 16), e(2, 0, 3, t=F), -torch.ones(3, device="cuda"),
                    e(2, 0, 1, 64), e(2, 0, 1, 64), S_in=S_in)
    assert y.shape == (2, 0, 3, 16)
    same(S, S_in, "state")
    _, S = ola.scan(e(2, 0, 3, 16), e(2, 0, 3, t=F), -torch.ones(3, device="cuda"),
                    e(2, 0, 1, 64), e(2, 0, 1, 64))
    assert bool((S == 0).all())
    st = gen(2, 3, 40, dtype=BF).cuda()
    y, s = ola.conv(e(2, 0, 40), gen(40, 4).cuda(), state=st)
    same(s, st, "window")


# ----------------------------------------------------------------------------- together

def _layer_inputs(R, P, H, d, seed):
    C = 3 * H * d
    return (gen(R, P, C, dtype=BF, seed=seed), gen(C, 4, seed=seed + 1, scale=0.5),
            gen(R, P, H, seed=seed + 2), gen(R, P, H, seed=seed + 3))


def _split(u, H, d):
    return [t.unflatten(2, (H, d)) for t in u.split(H * d, 2)]


@pytest.mark.gpu
def test_layer_prompt_then_beams():
    """Projections -> convolution -> unit queries and keys -> prefill, then two decode steps whose
    convolution windows follow the parents as the states do; against the 64-bit recurrence run on
    the same rounded queries, keys and values."""
    R, P, H, d, B, T = 2, 100, 2, 128, 6, 2
    x, w, g, b = _layer_inputs(R, P, H, d, 1)
    g, beta = -torch.nn.functional.softplus(g), torch.sigmoid(b)
    xc, wc = x.cuda(), w.cuda()
    u, win = ola.conv(xc, wc)
    q, k, v = _split(u, H, d)
    q, k = ola.qk_norm(q, k, l2=True)
    S = ola.prefill(k.contiguous(), v.contiguous(), g.cuda(), beta.cuda())
    # the definition, on what the operators rounded
    u64, _, tol = ref.conv(x, w, None, None, None, True, torch.zeros_like(x))
    close(u, u64, tol, "convolution")
    k64, kt = ref.qk_norm(_split(u.cpu(), H, d)[1].contiguous(), None, 1e-6, True, None, None, False)
    close(k, k64, kt, "keys")
    import numpy as np
    S64 = np.stack([[oracle.prefill(*(oracle.as_f64(t.cpu()[r, :, h]) for t in (k, v, g, beta)))
                     for h in range(H)] for r in range(R)])
    assert float((S.cpu().double() - torch.from_numpy(S64)).abs().max()) < 1e-4
    dec = ola.Decoder(S, B=B, T_max=T, in_dtype=BF)
    cur, parents, steps, outs = win[:, None], [], [], []
    for t in range(T):
        xs, _, gs, bs = _layer_inputs(R, B, H, d, 50 + 10 * t)
        gs, bs = -torch.nn.functional.softplus(gs), torch.sigmoid(bs)
        par = torch.zeros(R, B, dtype=torch.int32) if t == 0 else \
            torch.tensor([[0, 0, 3, 5, 5, 1], [2, 2, 2, 4, 0, 1]], dtype=torch.int32)
        us, cur = ola.conv_step(xs.cuda(), wc, state=cur, parent_idx=par.cuda())
        qs, ks, vs = _split(us, H, d)
        qs, ks = ola.qk_norm(qs, ks, l2=True)
        outs.append(dec.step(qs.contiguous(), ks.contiguous(), vs.contiguous(), gs.cuda(),
                             bs.cuda(), par.cuda()).cpu())
        steps.append([oracle.as_f64(y.cpu()) for y in (qs, ks, vs, gs, bs)])
        parents.append(par.numpy())
    want = oracle.decode_batch(S.double().cpu().numpy(),
                               *(np.stack([s[i] for s in steps]) for i in range(5)),
                               np.stack(parents))
    assert dec.error() == ola.OLA_OK and ola.layer_status() == ola.OLA_OK
    dec.close()
    assert float(np.abs(torch.stack(outs).double().numpy() - want).max()) <= 2e-3


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F])
def test_scan_prompt_then_steps_equals_longer_prompt(dtype):
    """The states of a prompt of P tokens, then n single tokens: the prompt of P + n tokens, up to
    what either form may lose."""
    R, P, n, H, G, dk, dv = 2, 130, 5, 2, 1, 64, 64
    c, o = _scan_case(dtype, R, P + n, H, G, dk, dv, z=True, D=True)
    y64, S64, ty, tS = ref.scan(**c, **{m: o[m] for m in ("D", "dt_bias", "z", "S_in", "lens")},
                                use_softplus=True, out0=torch.zeros(R, P + n, H, dv, dtype=dtype),
                                chunked=_chunked(dtype, dk))
    cg = {m: t.cuda() for m, t in c.items()}
    kw = dict(D=cu(o["D"]), dt_bias=cu(o["dt_bias"]))
    cut = lambda t, s: t if t.dim() == 1 else t[:, s].contiguous()  # noqa: E731
    head = {m: cut(t, slice(0, P)) for m, t in cg.items()}
    z = o["z"].cuda()
    y, S = ola.scan(**head, **kw, z=cut(z, slice(0, P)))
    ys, S = [y], S[:, None]
    for p in range(P, P + n):
        s = slice(p, p + 1)
        y, S = ola.scan_step(**{m: cut(t, s) for m, t in cg.items()}, **kw, z=cut(z, s), state=S)
        ys.append(y)
    close(torch.cat(ys, 1), y64, ty, "y")
    close(S[:, 0], S64, tS, "state")


@pytest.mark.gpu
def test_streams_and_graphs():
    """The calls run on the stream they are given, and a captured chain replays on new inputs, also
    while another captured chain with scratch of its own runs."""
    R, P, H, d = 1, 700, 2, 64
    c, o = _scan_case(BF, R, P, H, 1, d, d, bias=False)
    x, w = gen(R, P, H * d, dtype=BF, seed=11).cuda(), gen(H * d, 4, seed=12).cuda()
    cg = {m: t.cuda() for m, t in c.items()}

    def chain(x, k):
        u, _ = ola.conv(x, w)
        kk, qq = ola.qk_norm(k, cg["q"])
        return ola.scan(u.unflatten(2, (H, d)), cg["dt"], cg["A"], kk, qq)

    want = [chain(x, cg["k"]), chain(x * 2, cg["q"])]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, S = ola.scan(cg["v"], cg["dt"], cg["A"], cg["k"], cg["q"], stream=side)
    side.synchronize()
    y0, S0 = ola.scan(cg["v"], cg["dt"], cg["A"], cg["k"], cg["q"])
    same(y, y0, "y on another stream")
    same(S, S0, "state on another stream")
    graphs = []
    for i in range(2):
        xin, kin = torch.zeros_like(x), torch.zeros_like(cg["k"])
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            res = chain(xin, kin)
        graphs.append((gr, xin, kin, res))
    for i, (gr, xin, kin, res) in enumerate(graphs):
        xin.copy_(x * (i + 1))
        kin.copy_(cg["k"] if i == 0 else cg["q"])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for (gr, *_), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    for (_, _, _, res), wt in zip(graphs, want):
        same(res[0], wt[0], "y of a replay")
        same(res[1], wt[1], "state of a replay")
    assert ola.layer_status() == ola.OLA_OK


@pytest.mark.gpu
def test_results_do_not_change_from_run_to_run():
    c, o = _scan_case(BF, 2, 777, 4, 2, 128, 64, z=True, D=True)
    cg = {m: t.cuda() for m, t in c.items()}
    a = ola.scan(**cg, z=cu(o["z"]), D=cu(o["D"]))
    for _ in range(3):
        b = ola.scan(**cg, z=cu(o["z"]), D=cu(o["D"]))
        same(a[0], b[0], "y")
        same(a[1], b[1], "state")
