"""The entry points of include/kla_layer.h reject bad arguments on the host before anything is launched
(no GPU needed), and their workspace sizes are host calls."""
import pytest

# Fake, never dereferenced device addresses: every case below must be rejected on the host.
A = 0x7f0000000000
M = 0x10000000


@pytest.fixture(scope="module")
def lib():
    from gated_delta_rule_14_gb300 import _native, build
    build.build()
    return _native.lib()


def strides(*v):
    import ctypes
    return (ctypes.c_int64 * len(v))(*v)


def fwd(lib, **kw):
    a = dict(q=A, k=A + M, v=A + 2 * M, st=None, g=A + 3 * M, n=None, S0=None, o=A + 4 * M, ST=None, B=1, T=8, H=2,
             dk=16, dv=16, dt=0, s=1.0, ws=None, wb=0)
    a.update(kw)
    return lib.kla_linear_fwd(a["q"], a["k"], a["v"], a["st"], a["g"], a["n"], a["S0"], a["o"], a["ST"], a["B"],
                              a["T"], a["H"], a["dk"], a["dv"], a["dt"], a["s"], a["ws"], a["wb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), 1), (dict(g=None), 1), (dict(o=None), 1), (dict(B=0), 1), (dict(T=-1), 1), (dict(H=0), 1),
    (dict(dt=5), 1), (dict(s=float("nan")), 1), (dict(s=float("inf")), 1), (dict(dk=48), 2), (dict(dv=256), 2),
    (dict(q=A + 2), 1), (dict(q=A + 1, dt=1), 1), (dict(S0=A + 5 * M + 8), 1), (dict(ST=A + 5 * M + 4), 1),
    (dict(o=A), 1), (dict(ST=A + M), 1), (dict(n=A + 3), 1), (dict(st=strides(256, 32, -16, 256, 32, 16, 256, 32, 16)), 1),
    (dict(S0=A + 5 * M, ST=A + 5 * M + 16), 1),          # S_T over a part of S0
    (dict(T=100000, B=1, H=1), 1),                        # the segments' workspace is missing
    (dict(T=0, q=None, k=None, v=None, o=None), 0),       # nothing to do
])
def test_linear_fwd(lib, kw, code):
    assert fwd(lib, **kw) == code


def bwd(lib, **kw):
    a = dict(q=A, k=A + M, v=A + 2 * M, dO=A + 3 * M, st=None, g=A + 4 * M, n=None, S0=None, dST=None, dq=A + 5 * M,
             dk=A + 6 * M, dv=A + 7 * M, dS0=None, B=1, T=8, H=2, d_k=16, d_v=16, dt=0, s=1.0, ws=None, wb=0)
    a.update(kw)
    return lib.kla_linear_bwd(a["q"], a["k"], a["v"], a["dO"], a["st"], a["g"], a["n"], a["S0"], a["dST"], a["dq"],
                              a["dk"], a["dv"], a["dS0"], a["B"], a["T"], a["H"], a["d_k"], a["d_v"], a["dt"],
                              a["s"], a["ws"], a["wb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(dO=None), 1), (dict(dq=None), 1), (dict(dv=A), 1), (dict(dk=A + 5 * M), 1), (dict(dS0=A + 2), 1),
    (dict(dS0=A + 3 * M), 1), (dict(d_k=8), 2), (dict(s=float("nan")), 1), (dict(T=100000), 1),
    (dict(T=0, q=None, k=None, v=None, dO=None, dq=None, dk=None, dv=None), 0),
])
def test_linear_bwd(lib, kw, code):
    assert bwd(lib, **kw) == code


def test_linear_workspaces(lib):
    f, b = lib.kla_linear_fwd_workspace_size, lib.kla_linear_bwd_workspace_size
    assert f(64, 64, 16, 128, 128, 1) == 0                # enough chains: no segments
    assert f(1, 131072, 1, 128, 128, 1) > 0 and b(1, 131072, 1, 128, 128, 1) >= f(1, 131072, 1, 128, 128, 1)
    assert f(1, 0, 1, 128, 128, 1) == 0 and f(0, 5, 1, 128, 128, 1) == 0


def test_linear_step(lib):
    def call(**kw):
        a = dict(q=A, k=A + M, v=A + 2 * M, g=A + 3 * M, p=None, S=A + 4 * M, So=A + 4 * M, o=A + 5 * M, B=2, H=2,
                 dk=16, dv=16, N=2, dt=1, s=1.0)
        a.update(kw)
        return lib.kla_linear_step(a["q"], a["k"], a["v"], a["g"], a["p"], a["S"], a["So"], a["o"], a["B"], a["H"],
                                   a["dk"], a["dv"], a["N"], a["dt"], a["s"], None)
    assert call(S=None) == 1 and call(So=None) == 1 and call(q=A + 1) == 1 and call(S=A + 4 * M + 4) == 1
    assert call(N=3) == 1                                  # more states than sequences, and no parents
    assert call(p=A + 6 * M) == 1                          # parents, and the new states over the old
    assert call(So=A + 4 * M + 16) == 1 and call(So=A) == 1 and call(o=A + 4 * M) == 1
    assert call(dk=20) == 2 and call(s=float("inf")) == 1


def test_layer_norm(lib):
    def f(**kw):
        a = dict(x=A, w=A + M, b=A + 2 * M, y=A + 3 * M, m=A + 4 * M, r=A + 5 * M, rows=4, G=1, n=32, dt=1, eps=1e-5)
        a.update(kw)
        return lib.kla_layer_norm_fwd(a["x"], a["w"], a["b"], a["y"], a["m"], a["r"], a["rows"], a["G"], a["n"],
                                      a["dt"], a["eps"], None)
    assert f(x=None) == 1 and f(y=None) == 1 and f(rows=-1) == 1 and f(G=0) == 1 and f(n=0) == 1 and f(dt=9) == 1
    assert f(eps=-1.0) == 1 and f(eps=float("nan")) == 1 and f(eps=float("inf")) == 1 and f(y=A) == 1
    assert f(r=A + 4 * M) == 1 and f(n=2) == 2 and f(n=65537) == 2 and f(x=A + 1) == 1 and f(rows=0) == 0

    def g(**kw):
        a = dict(dy=A, x=A + M, w=A + 2 * M, m=A + 3 * M, r=A + 4 * M, dx=A + 5 * M, dw=A + 6 * M, db=A + 7 * M,
                 rows=4, G=1, n=32, dt=1, ws=A + 8 * M, wb=1 << 20)
        a.update(kw)
        return lib.kla_layer_norm_bwd(a["dy"], a["x"], a["w"], a["m"], a["r"], a["dx"], a["dw"], a["db"], a["rows"],
                                      a["G"], a["n"], a["dt"], a["ws"], a["wb"], None)
    assert g(dy=None) == 1 and g(m=None) == 1 and g(dx=A) == 1 and g(ws=None) == 1 and g(wb=16) == 1
    assert g(db=A + 6 * M) == 1 and g(ws=A + 8 * M + 8) == 1 and g(n=1) == 2
    assert lib.kla_layer_norm_bwd_workspace_size(0, 1, 32, 1) == 0


def test_beam(lib):
    def f(**kw):
        a = dict(x=A, ld=100, s=A + M, f=None, eos=-1, ns=A + 2 * M, p=A + 3 * M, t=A + 4 * M, nf=None, B=2, W=4,
                 V=100, dt=0, ws=A + 5 * M, wb=1 << 20)
        a.update(kw)
        return lib.kla_beam_select(a["x"], a["ld"], a["s"], a["f"], a["eos"], a["ns"], a["p"], a["t"], a["nf"],
                                   a["B"], a["W"], a["V"], a["dt"], a["ws"], a["wb"], None)
    assert f(x=None) == 1 and f(ws=None) == 1 and f(wb=8) == 1 and f(ld=99) == 1 and f(eos=100) == 1 and f(eos=-2) == 1
    assert f(f=A + 6 * M) == 1 and f(W=17) == 2 and f(W=0) == 1 and f(B=20000) == 2 and f(p=A + 2 * M) == 1
    assert f(ns=A + M) == 1 and f(dt=2) == 1 and f(x=A + 2) == 1 and f(V=3000000, ld=3000000) == 2
    r = lib.kla_reorder_states
    assert r(A, A + M, A, 1, 2, 64, None) == 1 and r(A, A + M, A + 2 * M, 1, 2, 24, None) == 1
    assert r(A, None, A + 2 * M, 1, 2, 64, None) == 1 and r(A + 8, A + M, A + 2 * M, 1, 2, 64, None) == 1
    assert r(A, A + M, A + 2 * M, 0, 2, 64, None) == 1 and r(A, A + M, A + 2 * M, 70000, 1, 64, None) == 2


def test_long_norm_rows_need_their_workspace(lib):
    """Rows of more than 8192 values keep two sums of each row in the workspace, wanted weights' gradients or
    not; its size is those sums, to 16 bytes, and the partial rows in front of which they lie."""
    def g(dw, ws, wb, n=9000, rows=3):
        return lib.kla_layer_norm_bwd(A, A + M, None, A + 2 * M, A + 3 * M, A + 4 * M, dw, None, rows, 1, n, 1, ws, wb,
                                      None)
    assert g(None, None, 0) == 1 and g(None, A + 8 * M, 31) == 1 and g(A + 6 * M, A + 8 * M, 32) == 1
    assert g(None, A, 32) == 1   # over dy
    size = lib.kla_layer_norm_bwd_workspace_size(3, 1, 9000, 1)
    assert size >= 32 + 2 * 9000 * 4 and (size - 32) % (2 * 9000 * 4) == 0
    assert g(A + 6 * M, A + 8 * M, size - 1) == 1


def test_team_selftest_rejects_its_arguments_on_host(lib):
    assert lib.kla_selftest_team_timeout(0, A, None) == 1 and lib.kla_selftest_team_timeout(100001, A, None) == 1
    assert lib.kla_selftest_team_timeout(10, None, None) == 1 and lib.kla_selftest_team_timeout(10, A + 2, None) == 1


def test_warp_selftest_rejects_its_arguments_on_host(lib):
    assert lib.kla_selftest_warp_timeout(0, A, None) == 1 and lib.kla_selftest_warp_timeout(100001, A, None) == 1
    assert lib.kla_selftest_warp_timeout(10, None, None) == 1 and lib.kla_selftest_warp_timeout(10, A + 2, None) == 1


FAR = 1 << 40   # buffers of tens of GB that do not overlap


@pytest.mark.parametrize("T", [2**31 - 1, 2**31 - 64, 2**31 - 65536])
def test_lengths_whose_chunks_pass_32_bits_are_refused(lib, T):
    """Tokens are numbered in 32 bits, up to the end of the last segment's last chunk."""
    q, k, v, g, o = (A + i * FAR for i in range(5))
    assert fwd(lib, q=q, k=k, v=v, g=g, o=o, T=T, H=1, dt=1, st=strides(*[0, 0, 16] * 3)) == 2
    a = [A + i * FAR for i in range(8)]
    assert bwd(lib, q=a[0], k=a[1], v=a[2], dO=a[3], g=a[4], dq=a[5], dk=a[6], dv=a[7], T=T, H=1, dt=1,
               st=strides(*[0, 0, 16] * 4)) == 2
    for size in (lib.kla_linear_fwd_workspace_size, lib.kla_linear_bwd_workspace_size):
        assert size(1, T, 1, 16, 16, 1) == 0 and size(1, T, 1, 128, 128, 1) == 0


@pytest.mark.parametrize("V", [2**31 - 1, 2**31 - 4000])
def test_vocabularies_whose_pieces_pass_32_bits_are_refused(lib, V):
    assert lib.kla_beam_select(A, V, A + FAR, None, -1, A + 2 * FAR, A + 3 * FAR, A + 4 * FAR, None, 1, 1, V, 1,
                               A + 5 * FAR, 1 << 39, None) == 2
    assert lib.kla_beam_select_workspace_size(1, 1, V, 1) == 0
