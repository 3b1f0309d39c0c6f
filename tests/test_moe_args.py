"""CPU: refusals and sizes of the grouped products, the fused epilogues and
the router (nothing here reaches a device)."""
import ctypes as C

import numpy as np
import pytest

from mlp_huffman_coded_b200 import synth
from mlp_huffman_coded_b200 import uw

from moe_util import act_f64, act_tail, activation_bound, route_ref

P = 0x10000  # a non-NULL, aligned address that no call may reach


@pytest.fixture(scope="module", autouse=True)
def built_library():
    from mlp_huffman_coded_b200 import build
    build.build()
    return uw.lib()


def table(n=4, rows=256, cols=512, ptr=P):
    t = uw.ExpertTable()
    t.n_experts, t.rows, t.cols, t.table = n, rows, cols, ptr
    return t


def matrix(rows=256, cols=512, pack=P):
    enc = uw.encode(synth.weight_matrix(rows, cols, 0.02, 1e-3, 100.0, 1))
    m = enc.matrix()
    m._keep = enc
    for f in ("sm", "stream", "chunk_bit_off", "vflags", "vprefix", "verbatim"):
        setattr(m, f, P)
    m.pack, m.pack_off = pack, pack
    return m


def test_structs_match_the_header():
    assert C.sizeof(uw.Epilogue) == 24
    assert C.sizeof(uw.ExpertTable) == 32
    assert uw.lib().uw_experts_table_bytes(3) == 3 * 80
    assert uw.lib().uw_experts_table_bytes(0) == 0
    assert uw.lib().uw_experts_table_bytes(1025) == 0


def test_workspace_sizes():
    f = uw.lib().uw_grouped_workspace_bytes
    t = table()
    one = f(C.byref(t), 8, 0)
    assert 0 < one < f(C.byref(t), 8, 1) and f(C.byref(t), 4096, 0) > one
    assert f(None, 8, 0) == 0 and f(C.byref(t), -1, 0) == 0
    assert f(C.byref(table(n=0)), 8, 0) == 0 and f(C.byref(table(n=2000)), 8, 0) == 0
    assert f(C.byref(table(cols=500)), 8, 0) == 0 and f(C.byref(table(cols=1 << 16)), 8, 0) == 0
    for n_rows in (1 << 30, (1 << 31) - 15, (1 << 31) - 1):
        assert f(C.byref(t), n_rows, 0) == f(C.byref(t), n_rows, 1) == 0
    # more units than an index holds
    assert f(C.byref(table(rows=1 << 20, cols=32768)), 1 << 22, 0) == 0
    g = uw.lib().uw_gemm_epilogue_workspace_bytes
    L = matrix().L
    assert g(C.byref(L), 1) > 0 and g(C.byref(L), 100000) > 0 and g(C.byref(L), -1) == 0 and g(None, 1) == 0


@pytest.mark.parametrize("n,rows,cols", [(1, 4096, 4096), (1, 14336, 4096), (8, 4096, 14336), (64, 2048, 1024),
                                         (8, 200, 192), (700, 1, 64)])
def test_a_workspace_for_more_rows_serves_fewer(n, rows, cols):
    lib = uw.lib()
    gate, down = table(n, rows, cols), table(n, 64 * -(-cols // 64), 64 * -(-rows // 64))
    up_to = [*range(1, 300), 511, 512, 513, 1000, 2048, 4096, 4097, 8192, 8193, 8256, 20000]
    for swiglu in (0, 1):
        sizes = [lib.uw_grouped_workspace_bytes(C.byref(gate), r, swiglu) for r in up_to]
        assert sizes[0] > 0 and sizes == sorted(sizes)
    L = uw.Layout()
    L.rows, L.cols = rows, cols
    sizes = [lib.uw_gemm_epilogue_workspace_bytes(C.byref(L), r) for r in up_to]
    assert sizes[0] > 0 and sizes == sorted(sizes)
    k = min(2, n)
    sizes = [lib.uw_moe_route_workspace_bytes(r, n, k) for r in up_to]
    assert sizes[0] > 0 and sizes == sorted(sizes)
    if rows % 64 == 0:
        sizes = [lib.uw_moe_workspace_bytes(C.byref(gate), C.byref(gate), C.byref(down), r, k) for r in up_to]
        assert sizes[0] > 0 and sizes == sorted(sizes)


@pytest.mark.parametrize("n,rows,cols", [(1, 200, 128), (1, 1, 64), (2, 64, 128), (8, 2048, 128), (64, 128, 512), (1024, 200, 128),
                                         (3, 4096, 4096)])
def test_every_batch_up_to_the_largest_is_taken(n, rows, cols):
    lib, most = uw.lib(), 1 << 22
    assert (most // 192 + n) * -(-rows // 128) * (cols // 64) < 1 << 31
    up_to = sorted({most, most - 1, *(int(1.07 ** i) for i in range(1, 226))})
    t, L = table(n, rows, cols), uw.Layout()
    L.rows, L.cols = rows, cols
    for swiglu in (0, 1):
        sizes = [lib.uw_grouped_workspace_bytes(C.byref(t), r, swiglu) for r in up_to]
        assert sizes[0] > 0 and sizes == sorted(sizes)
    sizes = [lib.uw_gemm_epilogue_workspace_bytes(C.byref(L), r) for r in up_to]
    assert sizes[0] > 0 and sizes == sorted(sizes)


def test_route_tensors_are_not_replaced():
    route = uw.Route(3, 4, 2, device="cpu")
    for name in ("weights", "experts", "slots", "rows", "offsets"):
        with pytest.raises(AttributeError):
            setattr(route, name, None)


def test_route_sizes():
    f = uw.lib().uw_moe_route_workspace_bytes
    assert f(1, 8, 2) > 0 and f(0, 8, 2) > 0 and f(1 << 20, 1024, 32) > 0
    for bad in ((-1, 8, 2), (1, 0, 1), (1, 8, 9), (1, 8, 0), (1, 64, 33), ((1 << 20) + 1, 8, 2), (1, 1025, 1)):
        assert f(*bad) == 0


@pytest.mark.parametrize("change", ["w", "offsets", "n_rows", "x_rows", "short_x", "table"])
def test_grouped_refusals(change):
    a = dict(w=C.byref(table()), x=P, x_rows=8, rows=None, offsets=P, n_rows=8)
    if change in ("w", "offsets"):
        a[change] = None
    elif change == "table":
        a["w"] = C.byref(table(ptr=P + 4))
    elif change == "short_x":
        a["x_rows"] = 7
    else:
        a[change] = -1
    st = uw.lib().uw_gemm_grouped(a["w"], a["x"], a["x_rows"], a["rows"], a["offsets"], a["n_rows"], None, P, P, 1 << 30,
                                  None)
    assert st == uw.UW_ERR_INVALID_ARG
    w = a["w"]
    st = uw.lib().uw_gemm_grouped_swiglu(w, w, a["x"], a["x_rows"], a["rows"], a["offsets"], a["n_rows"], P, P, 1 << 30,
                                         None)
    assert st == uw.UW_ERR_INVALID_ARG


def test_nothing_to_do_launches_nothing():
    n = uw.launch_count()
    t, m = table(), matrix()
    lib = uw.lib()
    assert lib.uw_gemm_grouped(C.byref(t), None, 0, None, P, 0, None, None, None, 0, None) == uw.UW_OK
    assert lib.uw_gemm_grouped_swiglu(C.byref(t), C.byref(t), None, 0, None, P, 0, None, None, 0, None) == uw.UW_OK
    assert lib.uw_gemm_epilogue(C.byref(m), None, 0, None, None, None, 0, None) == uw.UW_OK
    assert lib.uw_moe_combine(None, 1, None, None, 0, 2, 64, 0, None, None, None) == uw.UW_OK
    assert uw.launch_count() == n


def test_swiglu_gate_and_up_must_agree():
    for other in (table(n=3), table(rows=128), table(cols=256)):
        st = uw.lib().uw_gemm_grouped_swiglu(C.byref(table()), C.byref(other), P, 8, None, P, 8, P, P, 1 << 30, None)
        assert st == uw.UW_ERR_INVALID_ARG


def test_epilogue_refusals():
    lib = uw.lib()
    assert lib.uw_gemm_epilogue(None, P, 1, None, P, P, 1 << 30, None) == uw.UW_ERR_INVALID_ARG
    assert lib.uw_gemm_epilogue(C.byref(matrix()), P, -1, None, P, P, 1 << 30, None) == uw.UW_ERR_INVALID_ARG
    assert lib.uw_gemm_epilogue(C.byref(matrix(pack=None)), P, 1, None, P, P, 1 << 30, None) == uw.UW_ERR_INVALID_ARG


def test_experts_refusals():
    lib = uw.lib()
    a, b, out = matrix(), matrix(rows=128), uw.ExpertTable()

    def init(mats, n=None, ptr=P, nbytes=1 << 20):
        arr = (C.POINTER(uw.Matrix) * max(len(mats), 1))(*[C.pointer(m) if m else None for m in mats])
        return lib.uw_experts_init(arr, len(mats) if n is None else n, ptr, nbytes, C.byref(out), None)

    assert init([a, b]) == uw.UW_ERR_UNSUPPORTED_SHAPE
    assert init([a, matrix(pack=None)]) == uw.UW_ERR_INVALID_ARG
    assert init([a, None]) == uw.UW_ERR_INVALID_ARG
    assert init([a], n=0) == uw.UW_ERR_INVALID_ARG and init([a], n=1025) == uw.UW_ERR_INVALID_ARG
    assert init([a], ptr=None) == uw.UW_ERR_INVALID_ARG and init([a], ptr=P + 8) == uw.UW_ERR_INVALID_ARG
    assert init([a, a], nbytes=159) == uw.UW_ERR_WORKSPACE_TOO_SMALL
    a.cb.code_len[0] = 16
    assert init([a]) == uw.UW_ERR_CORRUPT
    with pytest.raises(uw.UwError):
        uw.Experts([])


def test_experts_init_allocates_nothing_that_could_throw(tmp_path):
    """Nothing throws across the ABI: with an operator new that fails, the
    call still returns a status (a child process, as a throw would end it)."""
    import os
    import subprocess
    import sys
    src, lib = tmp_path / "fail.cpp", tmp_path / "fail.so"
    src.write_text("""
        #include <cstdlib>
        #include <new>
        static bool fail = false;
        extern "C" void set_fail(int on) { fail = on; }
        void* operator new(std::size_t n) {
          void* p = fail ? nullptr : std::malloc(n);
          if (!p) throw std::bad_alloc();
          return p;
        }
        void operator delete(void* p) noexcept { std::free(p); }
        void operator delete(void* p, std::size_t) noexcept { std::free(p); }
    """)
    subprocess.run(["g++", "-shared", "-fPIC", "-O1", "-o", str(lib), str(src)], check=True)
    code = f"""
import ctypes as C, sys
sys.path[:0] = [{os.path.dirname(__file__)!r}, {os.path.dirname(os.path.dirname(uw.__file__))!r}]
from mlp_huffman_coded_b200 import uw
from test_moe_args import matrix, P
h, m, out = C.CDLL({str(lib)!r}), matrix(), uw.ExpertTable()
arr = (C.POINTER(uw.Matrix) * 1024)(*[C.pointer(m)] * 1024)
f = uw.lib().uw_experts_init
h.set_fail(1)
st = f(arr, 1024, P, 0, C.byref(out), None), f(arr, 1024, P + 8, 1 << 20, C.byref(out), None)
m.L.n_verbatim = -1  # refused before anything reaches a device
st += (f(arr, 1024, P, 1 << 20, C.byref(out), None),)
h.set_fail(0)
print(*st)
"""
    env = dict(os.environ, LD_PRELOAD=str(lib), CUDA_VISIBLE_DEVICES="")
    r = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-500:]
    assert r.stdout.split()[-3:] == [str(s) for s in (uw.UW_ERR_WORKSPACE_TOO_SMALL, uw.UW_ERR_INVALID_ARG, uw.UW_ERR_CORRUPT)]


def test_experts_keep_the_tensors_their_table_points_to(monkeypatch):
    """Preparing a matrix again replaces its pack; the table still holds the
    old one's address, so Experts has to keep it alive."""
    import gc
    import weakref

    import torch

    class Prepared:  # the parts of a DeviceMatrix that Experts takes
        class sm:
            get_device = staticmethod(lambda: 0)

        def __init__(self):
            self.mat = uw.Matrix()
            self.prepare_direct_palette()

        def prepare_direct_palette(self):
            self.pack, self.pack_off = torch.zeros(64, dtype=torch.uint8), torch.zeros(2, dtype=torch.int32)

    uw._need_torch()
    monkeypatch.setattr(uw, "_call", lambda *a: None)
    real = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **k: real(*a, **k))
    mats = [Prepared(), Prepared()]
    kept = [weakref.ref(t) for m in mats for t in (m.pack, m.pack_off)]
    ex = uw.Experts(mats)
    for m in mats:
        m.prepare_direct_palette()
    del m
    mats.clear()
    gc.collect()
    assert len(ex) == 2 and all(r() is not None for r in kept)
    del ex
    gc.collect()
    assert all(r() is None for r in kept)


def test_route_and_combine_refusals():
    lib = uw.lib()

    def route(logits=P, typ=1, T=4, E=8, k=2, w=P, off=P, ws=P, n=1 << 30):
        return lib.uw_moe_route(logits, typ, T, E, k, 1, w, P, P, P, off, ws, n, None)

    for bad in (dict(logits=None), dict(logits=P + 2), dict(typ=2), dict(T=-1), dict(E=0), dict(k=0), dict(k=9),
                dict(w=None), dict(off=None), dict(off=P + 2), dict(ws=None)):
        assert route(**bad) == uw.UW_ERR_INVALID_ARG, bad
    assert route(T=1000, n=256) == uw.UW_ERR_WORKSPACE_TOO_SMALL

    def combine(parts=P, typ=1, slots=P, w=P, T=4, k=2, cols=64, n=8, y=P):
        return lib.uw_moe_combine(parts, typ, slots, w, T, k, cols, n, None, y, None)

    for bad in (dict(parts=None), dict(parts=P + 2), dict(typ=5), dict(slots=None), dict(w=P + 2), dict(T=-1), dict(k=0),
                dict(k=33), dict(cols=0), dict(n=-1), dict(y=None)):
        assert combine(**bad) == uw.UW_ERR_INVALID_ARG, bad
    assert combine(cols=1 << 31) == uw.UW_ERR_UNSUPPORTED_SHAPE


def test_block_refusals():
    lib = uw.lib()
    g, u, d = table(rows=320, cols=256), table(rows=320, cols=256), table(rows=256, cols=320)
    need = lib.uw_moe_workspace_bytes(C.byref(g), C.byref(u), C.byref(d), 5, 2)
    assert need > 0
    for bad in ((g, u, g), (g, table(n=3, rows=320, cols=256), d), (g, table(rows=128, cols=256), d)):
        assert lib.uw_moe_workspace_bytes(*[C.byref(t) for t in bad], 5, 2) == 0
    assert lib.uw_moe_workspace_bytes(C.byref(g), C.byref(u), C.byref(d), 5, 5) == 0

    def block(gate=g, logits=P, typ=1, k=2, x=P, T=5, y=P, ws=P, n=need):
        return lib.uw_moe_block(C.byref(gate), C.byref(u), C.byref(d), logits, typ, k, 1, x, T, None, y, ws, n, None)

    for bad in (dict(gate=table(rows=128, cols=256)), dict(logits=None), dict(typ=7), dict(k=0), dict(x=None),
                dict(x=P + 2), dict(T=-1), dict(y=None), dict(ws=None)):
        assert block(**bad) == uw.UW_ERR_INVALID_ARG, bad
    assert block(n=need - 1) == uw.UW_ERR_WORKSPACE_TOO_SMALL
    assert block(T=0) == uw.UW_OK


def test_the_binding_checks_its_tensors():
    import torch
    uw._need_torch()
    good = torch.zeros(4, 8, dtype=torch.bfloat16)
    dev = good.get_device()  # -1: these live on the CPU
    assert uw._tensor(good, "t", uw._BF16, (4, 8), dev) == good.data_ptr()
    assert uw._tensor(good.view(torch.int16), "t", uw._BF16, (4, 8), dev) == good.data_ptr()
    assert uw._tensor(None, "t", uw._BF16, (4, 8), dev) is None
    for bad, types, shape, d in ((good, uw._BF16, (4, 9), dev), (good, uw._BF16, (32,), dev), (good, uw._FP32, (4, 8), dev),
                                 (good.t(), uw._BF16, (8, 4), dev), (good[:, ::2], uw._BF16, (4, 4), dev),
                                 (good, uw._BF16, (4, 8), 0)):
        with pytest.raises(uw.UwError) as e:
            uw._tensor(bad, "t", types, shape, d)
        assert e.value.status == uw.UW_ERR_INVALID_ARG
    for t in (None, torch.zeros(3), torch.zeros(2, 2, 2)):
        with pytest.raises(uw.UwError):
            uw._matrix_of(t, "t")
    with pytest.raises(uw.UwError):
        uw._out_type(torch.zeros(2, dtype=torch.float16), "t")
    with pytest.raises(uw.UwError):
        uw._epilogue(dev, (8,), 4, 8, good, None, "swish", None)
    # tensors that are on no CUDA device at all
    with pytest.raises(uw.UwError) as e:
        uw.moe_combine(torch.zeros(4, 8), torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2), good[:2].contiguous())
    assert e.value.status == uw.UW_ERR_INVALID_ARG


def test_counts_beyond_32_bits_are_not_wrapped(monkeypatch):
    """2^32 + 2 is not 2: the library's counts have 32 bits."""
    import torch
    uw._need_torch()
    big = 2**32 + 2
    L = matrix().L
    assert uw.route_workspace_bytes(2, 8, 2) > 0 and uw.epilogue_workspace_bytes(L, 2) > 0
    for n in (big, 2**31, 2**40, -big):
        assert uw.route_workspace_bytes(n, 8, 2) == uw.route_workspace_bytes(2, 8, n) == uw.route_workspace_bytes(2, n, 2) == 0
        assert uw.epilogue_workspace_bytes(L, n) == 0

    class Prepared:  # an Experts without a device
        device, rows, cols = -1, 320, 256

        def __init__(self, rows, cols):
            self.rows, self.cols, self.c = rows, cols, table(rows=rows, cols=cols)

        def __len__(self):
            return 4

    gate, down = Prepared(320, 256), Prepared(256, 320)
    assert uw.grouped_workspace_bytes(gate, 2) > 0 and uw.moe_workspace_bytes(gate, gate, down, 2, 2) > 0
    assert uw.grouped_workspace_bytes(gate, big) == 0
    assert uw.moe_workspace_bytes(gate, gate, down, big, 2) == uw.moe_workspace_bytes(gate, gate, down, 2, big) == 0

    monkeypatch.setattr(uw, "_call", lambda *a: pytest.fail("reached the library"))
    x, logits = torch.zeros(2, 256, dtype=torch.bfloat16), torch.zeros(2, 4)
    calls = [lambda: uw.moe_block(gate, gate, down, x, logits, big, x.clone(), None),
             lambda: uw.moe_block(gate, gate, down, x, None, 2, x.clone(), None),
             lambda: uw.moe_combine(torch.empty(big, 1, device="meta"), torch.zeros(2, 2, dtype=torch.int32),
                                    torch.zeros(2, 2), torch.zeros(2, 1, dtype=torch.bfloat16)),
             lambda: uw.Route(0, 8, big, device="cpu"),
             lambda: uw._matrix_of(torch.empty(big, 64, device="meta"), "x")]
    for i, call in enumerate(calls):
        with pytest.raises(uw.UwError) as e:
            call()
        assert e.value.status == uw.UW_ERR_INVALID_ARG, i


def test_the_plain_forms_themselves():
    """The references of the GPU tests at values worked by hand."""
    assert act_f64([-1.0, 2.0], "relu").tolist() == [0.0, 2.0]
    assert abs(act_f64([1.0], "gelu")[0] - 0.841344746068543) < 1e-14
    assert abs(act_f64([1.0], "gelu_tanh")[0] - 0.841191990608276) < 1e-14
    w, e, s, rows, off = route_ref(np.array([[0.0, 1.0, 1.0], [5.0, -np.inf, np.nan]], np.float32), 2)
    assert e.tolist() == [[1, 2], [0, -1]] and w.tolist() == [[0.5, 0.5], [1.0, 0.0]]
    assert s.tolist() == [[1, 2], [0, -1]] and rows.tolist() == [1, 0, 0] and off.tolist() == [0, 1, 2, 3]


def test_the_activations_bounds_tell_lost_tails_apart():
    """Forms that cancel, overflow or cut off for negative values break the
    bounds that the kernels' FP32 results are held to."""
    v = synth.bf16_bits_to_f32((np.arange(0x0080, 0x4300, dtype=np.uint16) | 0x8000))  # -2^-126 .. -128
    f, d = np.float32, v.astype(np.float64)
    from math import erf, pi, sqrt
    with np.errstate(all="ignore"):
        cancelling = {"gelu": f(0.5) * v * (f(1) + np.array([erf(t / sqrt(2)) for t in d], f)),
                      "gelu_tanh": f(0.5) * v * (f(1) + np.tanh(f(sqrt(2 / pi)) * (v + f(0.044715) * v * v * v))),
                      "silu": v / (f(1) + np.exp(-v))}  # exp overflows from -89 on
    for act, y in cancelling.items():
        ref, bound = act_tail(d, act), activation_bound(d, act)
        assert np.all(np.abs(ref.astype(f) - ref) <= bound)
        assert np.any(np.abs(y - ref) > bound), act
        cut = np.where(np.abs(ref) < 1e-36, 0.0, ref)
        assert np.any(np.abs(cut - ref) > bound), act
