"""ssm.h against the built library on a host without a GPU: every declared
function is exported, and every refusal of the documented calls comes back
with its status and a text before anything is enqueued."""
import ctypes
import os
import re

import pytest

from linear_attention_rnn_amd import ssm, wkv6

pytestmark = pytest.mark.skipif(not os.path.exists(wkv6.LIB_PATH), reason="libwkv6.so not built")

HEADER = os.path.join(os.path.dirname(wkv6.HEADER), "ssm.h")
A = 0x100000000   # fake, aligned addresses far apart: never dereferenced by a refused call
OK, INVALID, UNSUPPORTED, MISALIGNED = wkv6.OK, wkv6.ERR_INVALID_ARG, wkv6.ERR_UNSUPPORTED, wkv6.ERR_MISALIGNED


def P(i):
    return A * (i + 1)


def pointers(names, given):
    q = {n: P(i) for i, n in enumerate(names)}
    q.update(given)
    return q


def strides_of(s):
    return (ctypes.c_int64 * len(s))(*s) if s else None


def test_exports_and_version():
    with open(HEADER) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    names = set(re.findall(r"^\s*(?:int|size_t)\s+(ssm_\w+)\s*\(", text, flags=re.M))
    assert names == {"ssm_conv_fwd", "ssm_conv_bwd", "ssm_conv_bwd_workspace_bytes", "ssm_scan_fwd",
                     "ssm_scan_bwd", "ssm_scan_bwd_workspace_bytes", "ssm_block_norm",
                     "ssm_block_norm_bwd", "ssm_block_norm_bwd_workspace_bytes", "ssm_abi_version"}
    for n in names:
        assert ctypes.cast(getattr(ssm.lib(), n), ctypes.c_void_p).value
    value = lambda m: int(re.search(rf"#define {m}\s+(\d+)", text).group(1))  # noqa: E731
    assert ssm.abi_version() == value("SSM_ABI_VERSION") == 1
    assert (ssm.MAX_STATES, ssm.MAX_WINDOW, ssm.MAX_COLUMNS) == tuple(
        value(m) for m in ("SSM_MAX_STATES", "SSM_MAX_WINDOW", "SSM_MAX_COLUMNS"))
    assert {None: value("SSM_ACT_NONE"), "silu": value("SSM_ACT_SILU"), "sigmoid": value("SSM_ACT_SIGMOID")} == ssm._ACTIVATIONS


def refused(status, want, text=""):
    assert status == want, wkv6.last_error()
    assert wkv6.last_error() and text in wkv6.last_error()


# ---- ssm_conv_fwd, ssm_conv_bwd
def conv(B=2, T=9, D=64, W=4, act=1, dtype=1, strides=None, **p):
    q = pointers(("x", "weight", "bias", "lengths", "s_in", "y", "s_out"), p)
    return ssm.lib().ssm_conv_fwd(B, T, D, W, q["x"], q["weight"], q["bias"], act, q["lengths"], q["s_in"], q["y"],
                                  q["s_out"], strides_of(strides), dtype, 0)


def conv_bwd(B=2, T=9, D=64, W=4, act=1, dtype=1, strides=None, ws=(0, 0), **p):
    q = pointers(("x", "weight", "bias", "lengths", "s_in", "dy", "ds_out", "dx", "dweight", "dbias", "ds_in"), p)
    return ssm.lib().ssm_conv_bwd(B, T, D, W, q["x"], q["weight"], q["bias"], act, q["lengths"], q["s_in"], q["dy"],
                                  q["ds_out"], q["dx"], q["dweight"], q["dbias"], q["ds_in"], strides_of(strides), dtype, *ws, 0)


CONV = [(dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(D=0), INVALID), (dict(dtype=2), INVALID), (dict(act=2), INVALID),
        (dict(D=60), UNSUPPORTED), (dict(D=2 ** 20 + 8), UNSUPPORTED), (dict(W=1), UNSUPPORTED), (dict(W=5), UNSUPPORTED),
        (dict(B=2 ** 20), UNSUPPORTED), (dict(B=2 ** 62), UNSUPPORTED), (dict(T=2 ** 31), UNSUPPORTED),
        (dict(B=2 ** 10, T=2 ** 30), UNSUPPORTED), (dict(x=0), INVALID), (dict(weight=0), INVALID),
        (dict(x=P(0) + 4), MISALIGNED), (dict(weight=P(1) + 4), MISALIGNED), (dict(bias=P(2) + 4), MISALIGNED),
        (dict(lengths=P(3) + 4), MISALIGNED), (dict(s_in=P(4) + 8), MISALIGNED)]


@pytest.mark.parametrize("kw,want", CONV + [
    (dict(y=0), INVALID), (dict(y=P(5) + 2), MISALIGNED), (dict(s_out=P(6) + 4), MISALIGNED), (dict(y=P(0)), INVALID),
    (dict(y=P(0) + 64), INVALID), (dict(s_out=P(5)), INVALID), (dict(s_out=P(4) + 16), INVALID), (dict(y=P(3)), INVALID),
    (dict(strides=[-576, 64, 576, 64]), INVALID), (dict(strides=[576, 60, 576, 64]), MISALIGNED),
    (dict(strides=[576, 64, 576, 32]), INVALID), (dict(strides=[2 ** 62, 64, 576, 64]), UNSUPPORTED)])
def test_conv_refuses(kw, want):
    refused(conv(**kw), want)


@pytest.mark.parametrize("kw,want", CONV + [
    (dict(dy=0), INVALID), (dict(dx=0), INVALID), (dict(dweight=0), INVALID), (dict(dx=P(0)), INVALID), (dict(dx=P(5)), INVALID),
    (dict(dweight=P(1)), INVALID), (dict(dbias=P(8)), INVALID), (dict(ds_in=P(6)), INVALID), (dict(ds_in=P(10) + 4), MISALIGNED),
    (dict(strides=[576, 64, 576, 64, 0, 64]), INVALID), (dict(ws=(P(20), 8)), INVALID), (dict(ws=(P(20) + 4, 1 << 30)), MISALIGNED)])
def test_conv_bwd_refuses(kw, want):
    refused(conv_bwd(**kw), want)


def test_conv_without_work():
    assert conv(B=0, x=0, y=0, weight=0) == OK and conv(T=0, x=0, y=0, s_out=0) == OK
    refused(conv(T=0, s_out=P(4) + 16), INVALID, "s_out overlaps s_in")


# ---- ssm_scan_fwd, ssm_scan_bwd
SCAN = ("x", "dt", "A", "Bm", "Cm", "skip", "z", "dt_bias", "lengths", "s_in")


def scan(B=2, T=9, D=64, N=16, G=2, dtype=1, strides=None, **p):
    q = pointers(SCAN + ("y", "s_out"), p)
    a = [q[n] for n in SCAN]
    return ssm.lib().ssm_scan_fwd(B, T, D, N, G, *a[:8], 1, *a[8:], q["y"], q["s_out"], strides_of(strides), dtype, 0)


GRADS = ("dy", "ds_out", "dx", "ddt", "dA", "dB", "dC", "dskip", "dz", "ddt_bias", "ds_in")


def scan_bwd(B=2, T=9, D=64, N=16, G=2, dtype=1, strides=None, ws=(0, 0), **p):
    q = pointers(SCAN + GRADS, p)
    a = [q[n] for n in SCAN]
    return ssm.lib().ssm_scan_bwd(B, T, D, N, G, *a[:8], 1, *a[8:], *(q[n] for n in GRADS), strides_of(strides), dtype, *ws, 0)


CHANNELS, STATES = [9 * 64, 64, 0], [9 * 32, 32, 16]
ROWS = [*CHANNELS, *CHANNELS, *STATES, *STATES, *CHANNELS, *CHANNELS]
SIZES = [(dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(D=0), INVALID), (dict(G=0), INVALID), (dict(dtype=7), INVALID),
         (dict(D=60), UNSUPPORTED), (dict(G=3), UNSUPPORTED), (dict(G=16), UNSUPPORTED), (dict(N=0), UNSUPPORTED),
         (dict(N=12), UNSUPPORTED), (dict(N=72), UNSUPPORTED), (dict(B=2 ** 20), UNSUPPORTED), (dict(B=2 ** 60), UNSUPPORTED),
         (dict(T=2 ** 31), UNSUPPORTED),
         *((dict([(n, 0)]), INVALID) for n in ("x", "dt", "A", "Bm", "Cm")),
         *((dict([(n, P(i) + 4)]), MISALIGNED) for i, n in enumerate(SCAN))]


@pytest.mark.parametrize("kw,want", SIZES + [
    (dict(y=0), INVALID), (dict(y=P(10) + 8), MISALIGNED), (dict(s_out=P(11) + 4), MISALIGNED), (dict(y=P(0)), INVALID),
    (dict(y=P(6)), INVALID), (dict(y=P(3)), INVALID), (dict(s_out=P(10)), INVALID), (dict(s_out=P(9) + 16), INVALID),
    (dict(s_out=P(2)), INVALID), (dict(strides=[-576] + ROWS[1:]), INVALID), (dict(strides=ROWS[:7] + [28] + ROWS[8:]), MISALIGNED),
    (dict(strides=ROWS[:15] + [576, 32, 0]), INVALID), (dict(strides=ROWS[:6] + [2 ** 62] + ROWS[7:]), UNSUPPORTED)])
def test_scan_refuses(kw, want):
    refused(scan(**kw), want)


@pytest.mark.parametrize("kw,want", SIZES + [
    *((dict([(n, 0)]), INVALID) for n in ("dy", "dx", "ddt", "dA", "dB", "dC", "dz")), (dict(z=0), INVALID),
    *((dict([(n, P(10 + i) + 4)]), MISALIGNED) for i, n in enumerate(GRADS)),
    (dict(dx=P(0)), INVALID), (dict(ddt=P(12)), INVALID), (dict(dC=P(15)), INVALID), (dict(dz=P(6)), INVALID), (dict(dA=P(2)), INVALID),
    (dict(ds_in=P(9)), INVALID), (dict(ds_in=P(11) + 16), INVALID), (dict(dskip=P(5)), INVALID), (dict(ddt_bias=P(17)), INVALID),
    (dict(ws=(P(40), 64)), INVALID), (dict(ws=(P(40) + 8, 1 << 30)), MISALIGNED)])
def test_scan_bwd_refuses(kw, want):
    refused(scan_bwd(**kw), want)


def test_scan_without_work():
    none = {n: 0 for n in ("x", "dt", "Bm", "Cm", "z", "y")}
    assert scan(B=0, **none) == OK and scan(T=0, s_out=0, **none) == OK
    refused(scan(T=0, s_out=P(9) + 16, **none), INVALID, "s_out overlaps s_in")


# ---- ssm_block_norm, ssm_block_norm_bwd
def norm(rows=8, C=256, per=4, scale=1.0, act=1, eps=1e-5, dtype=1, **p):
    q = pointers(("x", "residual", "gate", "post", "pre", "h", "y"), p)
    return ssm.lib().ssm_block_norm(rows, C, q["x"], q["residual"], q["gate"], per, q["post"], q["pre"], scale, act, eps,
                                    q["h"], q["y"], dtype, 0)


def norm_bwd(rows=8, C=256, per=4, scale=1.0, act=1, eps=1e-5, dtype=1, ws=(0, 0), **p):
    q = pointers(("x", "h", "gate", "post", "pre", "dy", "dh", "dx", "dresidual", "dgate", "dpost", "dpre"), p)
    return ssm.lib().ssm_block_norm_bwd(rows, C, q["x"], q["h"], q["gate"], per, q["post"], q["pre"], scale, act, eps, q["dy"],
                                        q["dh"], q["dx"], q["dresidual"], q["dgate"], q["dpost"], q["dpre"], dtype, *ws, 0)


NORM = [(dict(rows=-1), INVALID), (dict(C=0), INVALID), (dict(C=100), UNSUPPORTED), (dict(C=16392), UNSUPPORTED),
        (dict(rows=2 ** 25 + 4), UNSUPPORTED), (dict(rows=2 ** 21 + 4, C=520), UNSUPPORTED), (dict(per=3), INVALID),
        (dict(per=0), INVALID), (dict(rows=2 ** 24, per=2, C=64), UNSUPPORTED), (dict(scale=float("inf")), INVALID), (dict(scale=float("nan")), INVALID),
        (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(act=3), INVALID), (dict(dtype=5), INVALID),
        (dict(gate=0), INVALID), (dict(x=0), INVALID), (dict(x=P(0) + 8), MISALIGNED), (dict(gate=P(2) + 4), MISALIGNED),
        (dict(post=P(3) + 4), MISALIGNED), (dict(pre=P(4) + 4), MISALIGNED), (dict(pre=0), INVALID)]


@pytest.mark.parametrize("kw,want", NORM + [
    (dict(h=0), INVALID), (dict(y=0), INVALID), (dict(residual=P(1) + 4), MISALIGNED), (dict(h=P(5) + 4), MISALIGNED),
    (dict(y=P(0)), INVALID), (dict(y=P(5)), INVALID), (dict(h=P(2)), INVALID), (dict(h=P(0) + 512), INVALID), (dict(y=P(4)), INVALID)])
def test_norm_refuses(kw, want):
    refused(norm(**kw), want)


@pytest.mark.parametrize("kw,want", NORM + [
    *((dict([(n, 0)]), INVALID) for n in ("h", "post", "dy", "dx", "dgate", "dpost", "dpre")),
    (dict(dx=P(0)), INVALID), (dict(dx=P(6)), INVALID), (dict(dresidual=P(5)), INVALID), (dict(dresidual=P(7)), INVALID),
    (dict(dgate=P(2)), INVALID), (dict(dpost=P(3)), INVALID), (dict(dpre=P(10)), INVALID), (dict(dx=P(5) + 512), INVALID),
    (dict(ws=(P(20), 64)), INVALID), (dict(ws=(P(20) + 4, 1 << 30)), MISALIGNED)])
def test_norm_bwd_refuses(kw, want):
    refused(norm_bwd(**kw), want)


def test_norm_without_rows():
    assert norm(rows=0) == OK


def test_workspace_bytes():
    assert ssm.conv_bwd_workspace_bytes(-1, 4, 64, 4) == 0 and ssm.conv_bwd_workspace_bytes(2, 100, 64, 4) >= 5 * 64 * 4
    assert ssm.scan_bwd_workspace_bytes(2, 100, 64, 12) == 0 and ssm.scan_bwd_workspace_bytes(2, 100, 64, 16) >= 2 * 64 * 16 * 4
    assert ssm.block_norm_bwd_workspace_bytes(10, 60) == 0
    assert ssm.block_norm_bwd_workspace_bytes(10, 64, 1, False, True, False) == 0   # a gate for every row needs no sums
    assert ssm.block_norm_bwd_workspace_bytes(10, 64, 5, False, True, False) >= 2 * 64 * 4
