"""The entry points of include/kla_block.h reject bad arguments on the host before anything is launched (no GPU
needed), and their workspace sizes are host calls."""
import ctypes

import pytest

# Fake, never dereferenced device addresses: every case below must be rejected on the host.
A = 0x7f0000000000
M = 0x10000000
FAR = 1 << 40   # buffers of tens of GB that do not overlap
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    from gated_delta_rule_14_gb300 import _native, build
    build.build()
    return _native.lib()


def strides(*v):
    return (ctypes.c_int64 * len(v))(*v)


def at(n):
    return [A + i * M for i in range(n)]


def scan(lib, **kw):
    x, g, y = at(3)
    a = dict(x=x, g=g, st=None, n=None, h0=None, y=y, hT=None, s=None, B=2, T=8, C=16, dt=0, mode=0, ws=A + 9 * M,
             wb=1 << 24)
    a.update(kw)
    return lib.kla_gated_scan_fwd(a["x"], a["g"], a["st"], a["n"], a["h0"], a["y"], a["hT"], a["s"], a["B"], a["T"],
                                  a["C"], a["dt"], a["mode"], a["ws"], a["wb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), 1), (dict(g=None), 1), (dict(y=None), 1), (dict(B=0), 1), (dict(T=-1), 1), (dict(C=0), 1),
    (dict(dt=5), 1), (dict(mode=2), 1), (dict(mode=-1), 1), (dict(x=A + 2), 1), (dict(g=A + M + 1, dt=1), 1),
    (dict(y=A), 1), (dict(y=A + M + 64), 1), (dict(n=A + 3), 1), (dict(h0=A + 3 * M + 2), 1),
    (dict(hT=A + 2 * M), 1), (dict(s=A), 1), (dict(st=strides(128, -16, 128, 16)), 1),
    (dict(h0=A + 3 * M, hT=A + 3 * M + 4), 1),              # h_T over a part of h0
    (dict(st=strides(M // 4, 16, 128, 16)), 1),             # x reaches into the gate's buffer, and y's
    (dict(T=2**31 - 1), 2), (dict(T=2**31 - 65536), 2), (dict(B=1 << 20), 2),
    (dict(C=2**31 - 1), 2), (dict(C=2**31 - 20, B=1, T=1), 2), (dict(B=65535, C=2**21, T=1000), 2),
    (dict(T=1000, ws=None, wb=0), 1), (dict(T=1000, wb=64), 1), (dict(T=1000, ws=A + 9 * M + 8), 1),
    (dict(T=1000, ws=A), 1),
])
def test_gated_scan_fwd(lib, kw, code):
    if kw.get("st") and code == 1 and kw["st"][0] == M // 4:
        kw = dict(kw, B=4)
    assert scan(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), 1), (dict(dy=None), 1), (dict(s=None), 1), (dict(dx=None), 1), (dict(dg=None), 1), (dict(dx=A), 1),
    (dict(dg=A + 4 * M), 1), (dict(dh0=A + 3 * M), 1), (dict(dhT=A + 6 * M + 1), 1), (dict(mode=7), 1),
    (dict(st=strides(128, 16, 128, 16, 128, -1)), 1), (dict(T=2**31 - 1), 2),
])
def test_gated_scan_bwd(lib, kw, code):
    p = at(6)
    a = dict(x=p[0], g=p[1], dy=p[2], st=None, n=None, s=p[3], dhT=None, dx=p[4], dg=p[5], dh0=None, B=2, T=8, C=16,
             dt=1, mode=1, ws=A + 9 * M, wb=1 << 24)
    a.update(kw)
    assert lib.kla_gated_scan_bwd(a["x"], a["g"], a["dy"], a["st"], a["n"], a["s"], a["dhT"], a["dx"], a["dg"],
                                  a["dh0"], a["B"], a["T"], a["C"], a["dt"], a["mode"], a["ws"], a["wb"], None) == code


def test_gated_scan_step(lib):
    def call(**kw):
        x, g, h, y = at(4)
        a = dict(x=x, xs=16, g=g, gs=16, h=h, y=y, B=2, C=16, dt=1, mode=0)
        a.update(kw)
        return lib.kla_gated_scan_step(a["x"], a["xs"], a["g"], a["gs"], a["h"], a["y"], a["B"], a["C"], a["dt"],
                                       a["mode"], None)
    assert call(x=None) == 1 and call(h=None) == 1 and call(xs=15) == 1 and call(gs=0) == 1 and call(C=0) == 1
    assert call(y=A) == 1 and call(y=A + 2 * M) == 1 and call(h=A + 2) == 1 and call(mode=3) == 1 and call(dt=2) == 1
    assert call(xs=M // 2, B=3) == 1                         # x's rows reach over the gate


def rotary(lib, **kw):
    q, k, oq, ok, f, p = at(6)
    a = dict(q=q, k=k, oq=oq, ok=ok, st=None, f=f, p=p, w=1, B=2, T=3, H=4, K=2, d=16, rot=8, lay=0, dt=1, s=1.0,
             inv=0)
    a.update(kw)
    return lib.kla_rotary(a["q"], a["k"], a["oq"], a["ok"], a["st"], a["f"], a["p"], a["w"], a["B"], a["T"], a["H"],
                          a["K"], a["d"], a["rot"], a["lay"], a["dt"], a["s"], a["inv"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(oq=None), 1), (dict(f=None), 1), (dict(rot=7), 1), (dict(rot=18), 1),
    (dict(rot=-2), 1), (dict(d=0, rot=0), 1), (dict(H=0), 1), (dict(K=-1), 1), (dict(B=-1), 1), (dict(lay=2), 1),
    (dict(dt=3), 1), (dict(s=NAN), 1), (dict(s=INF), 1), (dict(q=A + 1), 1), (dict(p=A + 5 * M + 4), 1),
    (dict(oq=A + 16), 1), (dict(oq=A + M), 1), (dict(ok=A + 2 * M), 1), (dict(oq=A + 4 * M), 1), (dict(d=1026), 2),
    (dict(B=1 << 16, T=1 << 16), 2), (dict(B=0), 0), (dict(T=0, q=None), 0),
    # one place for several of the output's values
    (dict(st=strides(192, 64, 16, 96, 32, 16, 192, 0, 16, 96, 32, 16)), 1),
    (dict(st=strides(192, 64, 16, 96, 32, 16, 192, 64, -16, 96, 32, 16)), 1),
    # an output over its input with other strides
    (dict(oq=A, st=strides(192, 64, 16, 96, 32, 16, 384, 64, 16, 96, 32, 16)), 1),
])
def test_rotary(lib, kw, code):
    assert rotary(lib, **kw) == code


@pytest.mark.parametrize("kw", [
    dict(k=A, oq=A, ok=A, K=4),                                        # queries and keys are one tensor, both in place
    dict(k=A, K=4, oq=A),                                              # the keys read what the queries write over
    dict(k=A + 3 * 16 * 4, oq=A),                                      # the keys start at the queries' last head
    dict(k=A + 64 * 4, K=4, oq=A, st=strides(192, 64, 16, 192, 64, 16, 192, 64, 16, 192, 64, 16)),   # a token later
    # slices of [2, 3, 5, 16], where the keys' two heads are the queries' last and the one behind
    dict(k=A + 3 * 16 * 4, oq=A, ok=A + 3 * 16 * 4, st=strides(240, 80, 16, 240, 80, 16, 240, 80, 16, 240, 80, 16)),
])
def test_rotary_of_queries_and_keys_that_share_values(lib, kw):
    assert rotary(lib, dt=0, **kw) == 1


def test_gated_norm(lib):
    def f(**kw):
        p = at(6)
        a = dict(x=p[0], g=p[1], gs=64, w=p[2], wg=1, y=p[3], m=p[4], r=p[5], rows=4, G=2, n=32, dt=1, norm=1, act=0,
                 eps=1e-5)
        a.update(kw)
        return lib.kla_gated_norm_fwd(a["x"], a["g"], a["gs"], a["w"], a["wg"], a["y"], a["m"], a["r"], a["rows"],
                                      a["G"], a["n"], a["dt"], a["norm"], a["act"], a["eps"], None)
    assert f(x=None) == 1 and f(g=None) == 1 and f(y=None) == 1 and f(gs=63) == 1 and f(rows=-1) == 1 and f(G=0) == 1
    assert f(norm=2) == 1 and f(act=2) == 1 and f(norm=0) == 1 and f(eps=-1.0) == 1 and f(eps=NAN) == 1
    assert f(y=A) == 1 and f(y=A + M) == 1 and f(r=A + 4 * M) == 1 and f(n=2) == 2 and f(n=65537, gs=1 << 20) == 2
    assert f(x=A + 1) == 1 and f(rows=0) == 0 and f(rows=1 << 31) == 2 and f(G=70000, gs=1 << 30) == 2
    assert f(gs=M // 2, rows=3) == 1                         # the gate's rows reach over the weights

    def b(**kw):
        p = at(9)
        a = dict(dy=p[0], x=p[1], g=p[2], gs=64, w=p[3], wg=1, m=None, r=p[4], dx=p[5], dg=p[6], dw=p[7], rows=4, G=2,
                 n=32, dt=1, act=0, ws=p[8], wb=1 << 24)
        a.update(kw)
        return lib.kla_gated_norm_bwd(a["dy"], a["x"], a["g"], a["gs"], a["w"], a["wg"], a["m"], a["r"], a["dx"],
                                      a["dg"], a["dw"], a["rows"], a["G"], a["n"], a["dt"], a["act"], a["ws"],
                                      a["wb"], None)
    assert b(dy=None) == 1 and b(r=None) == 1 and b(dx=None) == 1 and b(dg=None) == 1 and b(dx=A) == 1
    assert b(dg=A + 5 * M) == 1 and b(dw=A + 4 * M) == 1 and b(act=5) == 1 and b(gs=8) == 1 and b(n=1) == 2
    assert lib.kla_gated_norm_bwd_workspace_size(0, 2, 32, 1, 1) == 0
    need = lib.kla_gated_norm_bwd_workspace_size(4, 2, 32, 1, 1)
    assert need > 0 and b(ws=None, wb=need) == 1 and b(wb=need - 1) == 1 and b(ws=A) == 1
    assert b(ws=A + 8 * M + 8) == 1


def test_add_norm(lib):
    def f(**kw):
        p = at(8)
        a = dict(x=p[0], res=p[1], w=p[2], l=p[3], y=p[4], s=p[5], m=None, r=p[6], rows=4, n=32, dt=1, norm=0,
                 eps=1e-5)
        a.update(kw)
        return lib.kla_add_norm_fwd(a["x"], a["res"], a["w"], a["l"], a["y"], a["s"], a["m"], a["r"], a["rows"],
                                    a["n"], a["dt"], a["norm"], a["eps"], None)
    assert f(x=None) == 1 and f(res=None) == 1 and f(y=None) == 1 and f(s=None) == 1 and f(m=A + 7 * M) == 1
    assert f(s=A) == 1 and f(s=A + M + 16) == 1 and f(y=A + M) == 1 and f(y=A + 5 * M) == 1 and f(n=2) == 2
    assert f(eps=INF) == 1 and f(norm=3) == 1 and f(rows=0) == 0 and f(dt=4) == 1

    def b(**kw):
        p = at(12)
        a = dict(dy=p[0], ds=p[1], x=p[2], s=p[3], w=p[4], l=p[5], m=None, r=p[6], dx=p[7], dr=p[8], dw=p[9],
                 dl=p[10], rows=4, n=32, dt=1, ws=p[11], wb=1 << 24)
        a.update(kw)
        return lib.kla_add_norm_bwd(a["dy"], a["ds"], a["x"], a["s"], a["w"], a["l"], a["m"], a["r"], a["dx"],
                                    a["dr"], a["dw"], a["dl"], a["rows"], a["n"], a["dt"], a["ws"], a["wb"], None)
    assert b(dy=None) == 1 and b(s=None) == 1 and b(r=None) == 1 and b(dr=None) == 1 and b(dx=None) == 1
    assert b(x=None) == 1 and b(x=None, dl=None) == 1
    assert b(l=None) == 1 and b(l=None, dx=None) == 1 and b(l=None, dl=None) == 1
    assert b(dr=A + M) == 1 and b(dx=A + 8 * M) == 1 and b(dl=A + 9 * M) == 1 and b(n=2) == 2
    assert lib.kla_add_norm_bwd_workspace_size(0, 32, 1) == 0
    need = lib.kla_add_norm_bwd_workspace_size(4, 32, 1)
    assert need > 0 and b(ws=None, wb=need) == 1 and b(wb=need - 1) == 1 and b(ws=A) == 1


def test_verify_draft(lib):
    def f(**kw):
        p = at(7)
        a = dict(d=p[0], q=p[1], p=p[2], st=None, u=p[3], n=None, a=p[4], t=p[5], B=2, K=3, V=100, dt=0)
        a.update(kw)
        return lib.kla_verify_draft(a["d"], a["q"], a["p"], a["st"], a["u"], a["n"], a["a"], a["t"], a["B"], a["K"],
                                    a["V"], a["dt"], None)
    assert f(d=None) == 1 and f(p=None) == 1 and f(u=None) == 1 and f(a=None) == 1 and f(t=None) == 1 and f(B=0) == 1
    assert f(K=-1) == 1 and f(V=0) == 1 and f(dt=2) == 1 and f(a=A) == 1 and f(t=A + M) == 1 and f(t=A + 4 * M) == 1
    assert f(p=A + 2 * M + 2) == 1 and f(n=A + 6 * M + 1) == 1 and f(st=strides(300, -100, 400, 100)) == 1
    assert f(K=1025) == 2 and f(V=(1 << 24) + 1) == 2 and f(B=1 << 20) == 2


@pytest.mark.parametrize("T", [2**31 - 1, 2**31 - 64, 2**31 - 65536])
def test_lengths_whose_spans_pass_32_bits_are_refused(lib, T):
    assert scan(lib, x=A, g=A + FAR, y=A + 2 * FAR, B=1, T=T, C=1, dt=1, st=strides(0, 0, 0, 0)) == 2
    assert lib.kla_gated_scan_workspace_size(1, T, 1, 1) == 0
