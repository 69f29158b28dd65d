"""The operators around the recurrence at their edges: orderings that no result shows reliably, odd
calls that the documentation allows, and values at the ends of their types."""
import ctypes
import os
import re
import subprocess
import threading

import pytest
import torch

import layer_ref as ref
import linear_attention_beam_gdn_b200 as ola
from test_layer_ops import BF, F, SCAN, _chunked, _scan_case, close, cu, gen, same

CSRC = os.path.join(ola.PKG_DIR, "csrc")


# ----------------------------------------------------------------------------- chunked scan, order

def test_chunk_scan_waits_before_it_overwrites_the_weights():
    """Y1 reads the weights P from the tensor-memory columns that G of the next chunk is written to.
    The two products differ in shape and accumulator, so nothing orders them but a completion
    barrier: it has to be committed behind Y1 and waited for before G."""
    with open(os.path.join(CSRC, "ola_scan_chunk.cu")) as f:
        role = f.read().split("products Y1, G, Y2", 1)[1].split("// ----", 1)[0]
    y1, g = role.index("umma_bf16_ts(tmem + kTY1"), role.index("umma_bf16(tmem + kTG")
    assert y1 < g
    commit = re.search(r"umma_commit\((\w+)\)", role[y1:g])
    assert commit, "nothing tells when Y1 has read P"
    assert f"warp_wait({commit.group(1)}, i)" in role[y1 + commit.end():g]


@pytest.mark.gpu
@pytest.mark.parametrize("dk,H", [(128, 2), (64, 80)])
def test_scan_long_prompt(dk, H):
    """Thousands of tokens: in pieces of many chunks (few heads) and uncut; bit-equal from run to run."""
    R, P, dv = 1, 6000, 64
    c, o = _scan_case(BF, R, P, H, 1, dk, dv, D=True, state=True, seed=21)
    cg = {n: t.cuda() for n, t in c.items()}
    kw = dict(D=cu(o["D"]), dt_bias=cu(o["dt_bias"]), S_in=cu(o["S_in"]))
    y, S = ola.scan(**cg, **kw)
    assert ola.layer_status() == ola.OLA_OK
    for _ in range(5):
        y2, S2 = ola.scan(**cg, **kw)
        same(y2, y, "y")
        same(S2, S, "state")
    h = slice(0, 2)                                      # every head alone is the same recurrence
    y64, S64, ty, tS = ref.scan(c["v"][:, :, h], c["dt"][:, :, h], c["A"][h], c["k"], c["q"],
                                o["D"][h], o["dt_bias"][h], None, o["S_in"][:, h], None, True,
                                torch.zeros(R, P, 2, dv, dtype=BF), chunked=True)
    close(y[:, :, h], y64, ty, "y")
    close(S[:, h], S64, tS, "state")


# ----------------------------------------------------------------------------- values at the ends

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F, BF])
def test_silu_of_large_negative_values(dtype):
    """u / (1 + e^-u) goes to 0 below, however large u is; -inf and NaN give NaN, +inf itself."""
    u = torch.tensor([-3e38, -1e38, -1e30, -1e20, -1e6, -1000.0, -105.0, -104.0, -103.0, -89.0, -88.5,
                      -88.0, -87.0, -50.0, -1.0, 0.0, 1.0, 88.0, 1e30, 3e38, -float("inf"),
                      float("inf"), float("nan")]).to(dtype)
    x = u[None, None]
    w = torch.zeros(u.numel(), 2)
    w[:, 1] = 1.0
    y, _ = ola.conv(x.cuda(), w.cuda())
    u64 = u.double()
    want = u64 / (1 + torch.exp(-u64))
    y = y.cpu().double()[0, 0]
    assert torch.equal(torch.isnan(y), torch.isnan(want)), y
    inf = torch.isinf(want)
    assert torch.equal(y[inf], want[inf])
    # the steps of the division and the result's rounding; below -87, where fp32's exponent ends,
    # the result may be 0 or up to 104 e^-88 (6.3e-37)
    rel = 8 * 2.0 ** -24 if dtype == F else 2.0 ** -8 + 2.0 ** -20
    fine = ~torch.isnan(want) & ~inf
    assert bool(((y - want).abs()[fine] <= rel * want.abs()[fine] + 1.5e-36).all()), (y, want)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,P,H,lens", [(F, 130, 2, None), (F, 700, 1, [700, 333]),
                                            (BF, 130, 2, None), (BF, 130, 80, [130, 65]),
                                            (BF, 700, 1, [700, 333])])
def test_scan_infinite_decay(dtype, P, H, lens):
    """A = -inf forgets everything before each token; tokens behind a sequence's end (in the last
    tile of a prompt, too) decay nothing. The definition with A = -1e6 is the same: exp(-1e4) = 0."""
    R, dk, dv = 2, 64, 64
    c, o = _scan_case(dtype, R, P, H, 1, dk, dv, bias=False, softplus=False, state=True, lens=lens,
                      seed=31)
    c["dt"] = c["dt"] + 0.05
    c["A"][0] = -1e6
    out0 = torch.full((R, P, H, dv), 3.0, dtype=dtype)
    y64, S64, ty, tS = ref.scan(**c, D=None, dt_bias=None, z=None, S_in=o["S_in"], lens=o["lens"],
                                use_softplus=False, out0=out0, chunked=_chunked(dtype, dk))
    c["A"][0] = -float("inf")
    y, S = ola.scan(**{n: t.cuda() for n, t in c.items()}, S_in=cu(o["S_in"]), softplus=False,
                    lens=cu(o["lens"]), out=out0.cuda())
    assert ola.layer_status() == ola.OLA_OK
    close(y, y64, ty, "y")
    close(S, S64, tS, "state")


NAN, INF = float("nan"), float("inf")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,P,H,dk", [(BF, 200, 40, 128), (BF, 200, 40, 64), (BF, 1200, 2, 128),
                                          (F, 300, 2, 64), (F, 800, 1, 32), (BF, 200, 2, 256)])
@pytest.mark.parametrize("where", ["v", "k", "q", "dt", "z", "S_in", "decay"])
def test_scan_non_finite_inputs(dtype, P, H, dk, where):
    """A value that is not finite makes exactly those outputs and state elements not finite that the
    formula makes so; all others are as good as ever."""
    R, dv, G = 2, 64, 1
    c, o = _scan_case(dtype, R, P, H, G, dk, dv, z=True, state=True, bias=False, softplus=False,
                      lens=[P, P - 70], seed=41)
    at = [(0, 10), (0, 140), (1, 127), (1, 63)]
    for i, (r, p) in enumerate(at):
        bad = (NAN, INF, -INF, NAN)[i]
        h, e = i % H, (7 * i) % dv
        if where in ("v", "z"):
            (c if where == "v" else o)[where][r, p, h, e] = bad
        elif where in ("k", "q"):
            c[where][r, p, 0, (9 * i) % dk] = bad
        elif where == "dt":
            c["dt"][r, p, h] = abs(bad)
        elif where == "S_in":
            o["S_in"][r, h, e, (9 * i) % dk] = bad
    if where == "decay":                                  # 0 * -inf: not a number from there on
        c["A"][0] = -INF
        c["dt"] = c["dt"] + 0.05
        c["dt"][0, 140, 0] = c["dt"][1, 20, 0] = 0.0
    out0 = torch.full((R, P, H, dv), 3.0, dtype=dtype)
    want = dict(c)
    if where == "decay":
        # the bound is not made for an infinite A: this head is compared by where it is finite only
        want["A"] = c["A"].clone()
        want["A"][0] = -1e6
    y64, S64, ty, tS = ref.scan(**want, D=None, dt_bias=None, z=o["z"], S_in=o["S_in"], lens=o["lens"],
                                use_softplus=False, out0=out0, chunked=_chunked(dtype, dk))
    if where == "decay":
        y64[0, 140:, 0], S64[0, 0] = NAN, NAN
        y64[1, 20:P - 70, 0], S64[1, 0] = NAN, NAN
    y, S = ola.scan(**{n: t.cuda() for n, t in c.items()}, z=cu(o["z"]), S_in=cu(o["S_in"]),
                    lens=cu(o["lens"]), softplus=False, out=out0.cuda())
    assert ola.layer_status() == ola.OLA_OK
    for got, w64, tol, what in ((y, y64, ty, "y"), (S, S64, tS, "state")):
        got, fine = got.cpu().double(), torch.isfinite(w64)
        assert torch.equal(torch.isfinite(got), fine), \
            (what, (torch.isfinite(got) & ~fine).nonzero()[:4], (~torch.isfinite(got) & fine).nonzero()[:4])
        zero = torch.zeros_like(w64)
        close(torch.where(fine, got, zero), torch.where(fine, w64, zero),
              torch.where(fine, tol, zero + 1), what)


def _time(fn, n=5):
    fn()
    ts = []
    for _ in range(n):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        fn()
        b.record()
        b.synchronize()
        ts.append(a.elapsed_time(b))
    return min(ts)


@pytest.mark.gpu
@pytest.mark.parametrize("cols", [1, 64])
def test_scan_late_bad_value_costs_a_second_look_not_a_walk(cols):
    """The outputs before a value that is not finite, in its own chunk, are taken again from the
    state before the chunk. That is work of the order of the call itself."""
    R, P, H, dk, dv = 1, 5120, 40, 128, 128
    c, _ = _scan_case(BF, R, P, H, 1, dk, dv, bias=False, seed=51)
    cg = {n: t.cuda() for n, t in c.items()}
    out, S = torch.empty_like(cg["v"]), torch.empty(R, H, dv, dk, device="cuda")
    clean = _time(lambda: ola.scan(**cg, out=out, S_out=S))
    y0 = out.clone()
    p = 5000
    cg["v"][0, p, 3, :cols] = NAN
    dirty = _time(lambda: ola.scan(**cg, out=out, S_out=S))
    assert not torch.isfinite(out[0, p:, 3, :cols]).any()
    h = slice(3, 4)
    y64, _, ty, _ = ref.scan(c["v"][:, :p, h], c["dt"][:, :p, h], c["A"][h], c["k"][:, :p],
                             c["q"][:, :p], None, None, None, None, None, True,
                             torch.zeros(R, p, 1, dv, dtype=BF), chunked=True)
    close(out[:, :p, h], y64, ty, "y before it")
    y0[0, :, 3, :cols] = out[0, :, 3, :cols] = 0.0
    same(out, y0, "y elsewhere")
    print(f"clean {clean * 1e3:.0f} us, one bad token in {cols} columns {dirty * 1e3:.0f} us")
    assert dirty <= 16 * clean, (clean, dirty)


# ----------------------------------------------------------------------------- calls of every kind

@pytest.mark.gpu
@pytest.mark.parametrize("R", [1, 3])
def test_one_token_slices_of_one_buffer(R):
    """One token of each of R requests: inputs and outputs are column slices of one buffer."""
    H, d, W = 2, 32, 4
    C = H * d
    buf = gen(R, 1, 7 * C, dtype=BF, seed=61).cuda()
    part = lambda i: buf[:, :, i * C:(i + 1) * C]  # noqa: E731
    heads = lambda i: part(i).unflatten(2, (H, d))  # noqa: E731
    w, win = gen(C, W, seed=62).cuda(), gen(R, 1, W - 1, C, dtype=BF, seed=63).cuda()
    y0, s0 = ola.conv_step(part(0).contiguous(), w, state=win)
    y1, s1 = ola.conv_step(part(0), w, state=win, out=part(4))
    same(part(4).contiguous(), y0, "convolution step")
    same(s1, s0, "window")
    ola.conv(part(0), w, state=win[:, 0].contiguous(), out=part(5))
    same(part(5).contiguous(), y0, "convolution")
    dt, A = gen(R, 1, H, seed=64).cuda(), -torch.ones(H).cuda()
    S = gen(R, 1, H, d, d, seed=65).cuda()
    args = [heads(i).contiguous() for i in (1, 2, 3)]
    y0, S0 = ola.scan_step(args[0], dt, A, args[1], args[2], state=S)
    _, S1 = ola.scan_step(heads(1), dt, A, heads(2), heads(3), state=S, out=heads(6))
    same(heads(6).contiguous(), y0, "scan step")
    same(S1, S0, "state")
    y0, S0 = ola.scan(args[0], dt, A, args[1], args[2], S_in=S[:, 0].contiguous())
    ola.scan(heads(1), dt, A, heads(2), heads(3), S_in=S[:, 0].contiguous(), out=heads(4))
    same(heads(4).contiguous(), y0, "scan")
    for i in (1, 2, 3):                                   # a real overlap is still refused
        with pytest.raises(ola.OlaError):
            ola.scan_step(heads(1), dt, A, heads(2), heads(3), state=S, out=heads(i))


@pytest.mark.gpu
def test_status_reports_every_error_once():
    """Threads that read the error word on streams of their own: each recorded error is returned to
    exactly one of them."""
    # one beam of 8 bf16 channels: one device thread reads the parent, so a call records one error
    x, w, st = gen(1, 1, 8, dtype=BF).cuda(), gen(8, 4, seed=1).cuda(), \
        gen(1, 1, 3, 8, dtype=BF, seed=3).cuda()
    bad = torch.tensor([[4]], dtype=torch.int32).cuda()
    assert ola.layer_status() == ola.OLA_OK
    torch.cuda.synchronize()
    L, n, stop, seen = ola.lib(), 1000, threading.Event(), [0, 0, 0]

    def poll(i):
        side = torch.cuda.Stream()
        while not stop.is_set():
            for _ in range(50):
                seen[i] += L.ola_layer_status(side.cuda_stream) == ola.OLA_ERR_BAD_PARENT

    threads = [threading.Thread(target=poll, args=(i,)) for i in (1, 2)]
    for t in threads:
        t.start()
    here = torch.cuda.current_stream().cuda_stream
    try:
        for _ in range(n):
            ola.conv_step(x, w, state=st, parent_idx=bad)
            seen[0] += L.ola_layer_status(here) == ola.OLA_ERR_BAD_PARENT
    finally:
        stop.set()
        for t in threads:
            t.join()
    assert sum(seen) == n and ola.layer_status() == ola.OLA_OK, seen


def test_refuses_a_stream_of_another_device():
    """Kernels would run on the stream's device with pointers of another one."""
    class Stream:
        device_index = 1
        device = torch.device("cuda", 1)
        cuda_stream = 0

    with pytest.raises(ValueError, match="stream"):
        ola._scope(0, Stream())
    for device in (0, "cuda:0", torch.device("cuda", 0)):
        with pytest.raises(ValueError, match="stream"):
            ola.layer_status(device, Stream())


# ----------------------------------------------------------------------------- strides and overlaps

DRIVER = r"""
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "ola_rows.h"

int main(int n, char** v) {
  int64_t x[16] = {};
  for (int i = 2; i < n && i < 18; ++i) x[i - 2] = strtoll(v[i], nullptr, 0);
  auto rows = [&](int i) {
    return ola::Rows{reinterpret_cast<const void*>(x[i]), x[i + 1], x[i + 2], x[i + 3], x[i + 4],
                     x[i + 5], int(x[i + 6])};
  };
  if (!strcmp(v[1], "overlap")) {
    ola::Rows a = rows(0), b = rows(7);
    if (!ola::strides(&a, false) || !ola::strides(&b, true)) return 2;
    printf("%d", ola::overlap(a, b));
  } else if (!strcmp(v[1], "strides")) {
    ola::Rows a = rows(0);
    printf("%d", ola::strides(&a, x[7]));
  }
}
"""


@pytest.fixture(scope="module")
def rows(tmp_path_factory):
    """The library's checks of row tensors, compiled so that a signed overflow ends the process."""
    d = tmp_path_factory.mktemp("rows")
    (d / "rows.cpp").write_text(DRIVER)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=signed-integer-overflow",
                    "-fsanitize-undefined-trap-on-error", "-I", CSRC, "-o", str(d / "rows"),
                    str(d / "rows.cpp")], check=True)

    def call(what, *args):
        p = subprocess.run([str(d / "rows"), what, *map(str, args)], capture_output=True, text=True)
        assert p.returncode == 0, (what, args, p.returncode)
        return int(p.stdout)

    return call


@pytest.mark.parametrize("R,P", [(1, 1), (3, 1), (1, 4), (3, 4)])
def test_overlap_of_column_slices(rows, R, P):
    """Column slices of one [R, P, wide] buffer share bytes where their columns do, also with one
    token per sequence, where the token stride is not used."""
    wide, e, base = 700, 2, 1 << 20

    def at(col, width):
        tok = wide if P > 1 else 0                        # as the Python binding passes them
        return (base + col * e, R, P, tok, P * wide, width, e)

    # column, width of an input; of the output
    for i, o, want in (((0, 100), (100, 100), 0), ((100, 100), (0, 100), 0), ((0, 100), (600, 100), 0),
                       ((0, 64), (100, 100), 0), ((500, 100), (100, 400), 0), ((0, 100), (99, 100), 1),
                       ((100, 100), (0, 101), 1), ((0, 700), (300, 10), 1), ((300, 10), (0, 700), 1),
                       ((0, 100), (0, 100), 1)):
        assert rows("overlap", *at(*i), *at(*o)) == want, (i, o)
    # another buffer behind the first, and one that starts inside it
    behind = (base + R * P * wide * e, R, P, 0, 0, 100, e)
    inside = (base + 50 * e, 1, 1, 0, 0, 100, e)
    assert rows("overlap", *at(0, 100), *behind) == 0
    assert rows("overlap", *at(0, 100), *inside) == 1


@pytest.mark.parametrize("R,P,tok,seq,output", [
    (2, 5, 1 << 62, 0, 0), (2, 5, 1 << 62, 0, 1), (2, 5, 1 << 62, 100, 1), (2, 3, 1 << 45, 0, 1),
    (1 << 30, 2, 0, 1 << 40, 1), (1, 1 << 30, 1 << 40, 0, 0), (2, 1, 0, (1 << 63) - 1, 1)])
def test_strides_too_large_are_refused_without_overflow(rows, R, P, tok, seq, output):
    assert rows("strides", 1 << 20, R, P, tok, seq, 16, 4, output) == 0


def test_refuses_more_elements_than_64_bits_hold():
    """Products of sizes past 2^46, the state counts of a step among them, are refused, not wrapped."""
    L, far = ola.lib(), [(i + 1) << 52 for i in range(12)]
    top = (1 << 31) - 1
    c = ola.ConvDesc(top, 0, top, 4, ola.OLA_F32, 1, 0, 0, 0, 0)
    assert L.ola_conv(ctypes.byref(c), *far[:7], None) == ola.OLA_ERR_UNSUPPORTED
    c = ola.ConvDesc(1 << 16, 1, 1 << 16, 4, ola.OLA_F32, 1, 0, 0, 0, 0)
    assert L.ola_conv_step(ctypes.byref(c), top, *far[:4], far[4], *far[5:7], None) == \
        ola.OLA_ERR_UNSUPPORTED
    d = ola.ScanDesc(1 << 12, 1, 1 << 12, 1, 256, 256, ola.OLA_F32, 1, *[0] * 10)
    assert L.ola_scan_step(ctypes.byref(d), top, *far, None) == ola.OLA_ERR_UNSUPPORTED


# ----------------------------------------------------------------------------- alignments

@pytest.mark.gpu
@pytest.mark.parametrize("dtype,C,off,wide", [(BF, 64, 4, 72), (BF, 66, 2, 132), (BF, 1000, 4, 1004),
                                              (BF, 6, 2, 10), (F, 18, 2, 22), (F, 64, 2, 66)])
@pytest.mark.parametrize("W", [2, 4])
def test_conv_rows_aligned_to_8_and_4_bytes(dtype, C, off, wide, W):
    R, P = 3, 61
    big = gen(R, P, wide, dtype=dtype, seed=71)
    w, b = gen(C, W, seed=72), gen(C, seed=73)
    st = gen(R, W - 1, C, dtype=dtype, seed=74)
    lens = torch.tensor([61, 1, 40], dtype=torch.int32)
    out0 = torch.full((R, P, C), 3.0, dtype=dtype)
    x = big[:, :, off:off + C]
    y64, s64, tol = ref.conv(x.contiguous(), w, b, st, lens, True, out0)
    y, s = ola.conv(big.cuda()[:, :, off:off + C], w.cuda(), b.cuda(), state=st.cuda(),
                    lens=lens.cuda(), out=out0.cuda())
    close(y, y64, tol, "y")
    assert torch.equal(s.cpu().double(), s64)


@pytest.mark.gpu
@pytest.mark.parametrize("R,P,H,G,dk,dv,opt", [s[1:] for s in SCAN if s[0] == BF])
def test_scan_rows_off_16_bytes(R, P, H, G, dk, dv, opt):
    """bf16 rows that start off a 16-byte boundary run token by token in fp32: the definition within
    the bounds of fp32 sums."""
    c, o = _scan_case(BF, R, P, H, G, dk, dv, **opt)
    sp = opt.get("softplus", True)
    out0 = torch.full((R, P, H, dv), 3.0, dtype=BF)
    y64, S64, ty, tS = ref.scan(**c, D=o["D"], dt_bias=o["dt_bias"], z=o["z"], S_in=o["S_in"],
                                lens=o["lens"], use_softplus=sp, out0=out0, chunked=False)

    def odd(t):
        if t is None:
            return None
        room = torch.zeros(t.numel() + 8, device="cuda", dtype=BF)
        x = room[1:1 + t.numel()].view(t.shape)
        assert x.data_ptr() % 16 == 2
        return x.copy_(t)

    cg = {n: odd(t) if n in ("v", "k", "q") else t.cuda() for n, t in c.items()}
    y, S = ola.scan(**cg, D=cu(o["D"]), dt_bias=cu(o["dt_bias"]), z=odd(o["z"]), S_in=cu(o["S_in"]),
                    lens=cu(o["lens"]), softplus=sp, out=odd(out0))
    assert ola.layer_status() == ola.OLA_OK
    close(y, y64, ty, "y")
    close(S, S64, tS, "state")
