"""Refusals of the calls over a paged cache: every call below is rejected by the host checks before
any CUDA call is made, so they run without a GPU."""

import ctypes

import pytest
import torch

P, L, F = ctypes.c_void_p, ctypes.c_longlong, ctypes.c_float
NULL = P(0)


def at(i, off=0):
    """Addresses 1 TiB apart: nothing overlaps unless a case asks for it."""
    return P(((i + 1) << 40) + off)


@pytest.fixture(scope="module")
def lib():
    from conftest import load_builder
    return ctypes.CDLL(load_builder().build())


def tables_args(**o):
    return [o.get("lens", at(0)), o.get("news", at(1)), o.get("B", 4), o.get("table", at(2)), o.get("width", 10),
            o.get("stack", at(3)), o.get("pages", 100), o.get("n_free", at(4)), o.get("page", 16), o.get("T", 8),
            o.get("starts", at(5)), o.get("positions", at(6)), o.get("slots", at(7)), o.get("lens_out", at(8)),
            o.get("n_free_out", at(9)), NULL]


def test_page_tables_refusals(lib):
    f = lib.rf_page_tables
    names = ("lens", "news", "table", "stack", "n_free", "starts", "positions", "slots", "lens_out", "n_free_out")
    for name in names:
        assert f(*tables_args(**{name: NULL})) == 1, name
    for name in ("B", "width", "pages", "page", "T"):
        assert f(*tables_args(**{name: 0})) == 1, name
        assert f(*tables_args(**{name: -3})) == 1, name
    assert f(*tables_args(B=8193)) == 2
    assert f(*tables_args(B=8192, width=1 << 18)) == 2
    assert f(*tables_args(pages=1 << 27)) == 2
    assert f(*tables_args(width=1 << 27, B=1)) == 2
    for name in ("positions", "slots"):
        assert f(*tables_args(**{name: at(20, 4)})) == 3, name
    # outputs on inputs or on one another; lens_out may only be lens itself, n_free_out n_free
    for name in ("table", "stack", "starts", "positions", "slots", "lens_out", "n_free_out"):
        assert f(*tables_args(**{name: at(1)})) == 1, name
    assert f(*tables_args(lens_out=at(0, 4))) == 1
    assert f(*tables_args(lens_out=at(4))) == 1
    assert f(*tables_args(slots=at(6, 16))) == 1
    assert f(*tables_args(starts=at(3, 396))) == 1


def rope_args(**o):
    return [o.get("q", at(0)), L(o.get("q_step", 1024)), o.get("k", at(1)), L(o.get("k_step", 256)),
            o.get("v", at(2)), L(o.get("v_step", 256)), o.get("T", 5), o.get("H", 8), o.get("Hkv", 2),
            o.get("D", 128), o.get("qw", NULL), NULL, o.get("w_dtype", 1), F(o.get("eps", 1e-6)),
            o.get("positions", at(3)), o.get("axes", 1), o.get("freq", at(4)), NULL, o.get("R", 128), 0,
            o.get("dtype", 1), o.get("slots", at(5)), o.get("pages", 10), o.get("page", 16),
            o.get("q_out", at(6)), o.get("k_out", at(7)), o.get("v_out", at(8)), NULL]


def test_norm_rope_refusals(lib):
    f = lib.rf_qk_norm_rope
    for name in ("q", "k", "v", "positions", "freq", "slots", "q_out", "k_out", "v_out"):
        assert f(*rope_args(**{name: NULL})) == 1, name
    for name in ("T", "H", "Hkv", "D", "axes", "R", "pages", "page"):
        assert f(*rope_args(**{name: 0})) == 1, name
        assert f(*rope_args(**{name: -16})) == 1, name
    assert f(*rope_args(R=144)) == 1                # more than D
    assert f(*rope_args(R=24)) == 2
    assert f(*rope_args(D=96, R=96, q_step=768)) == 2
    assert f(*rope_args(D=512, q_step=1 << 13, k_step=1 << 13, v_step=1 << 13)) == 2
    assert f(*rope_args(dtype=0, w_dtype=0)) == 2   # fp32 rows
    assert f(*rope_args(dtype=3, w_dtype=0)) == 1
    assert f(*rope_args(w_dtype=2)) == 1            # fp16 weights of bf16 rows
    for eps in (-1.0, float("nan"), float("inf")):
        assert f(*rope_args(eps=eps)) == 1
    for name in ("q_step", "k_step", "v_step"):
        assert f(*rope_args(**{name: 248})) == 1, name          # shorter than a row
        assert f(*rope_args(**{name: 1028})) == 3, name
        assert f(*rope_args(**{name: 1 << 41})) == 2, name
    for name in ("q", "k", "v", "q_out", "k_out", "v_out"):
        assert f(*rope_args(**{name: at(20, 8)})) == 3, name
    assert f(*rope_args(T=(1 << 31) - 1)) == 2
    assert f(*rope_args(pages=1 << 27)) == 2


@pytest.mark.skipif(torch.cuda.is_available(), reason="a call that is not refused would be launched")
def test_norm_rope_refuses_overlapping_buffers(lib):
    """Outputs over rows that other warps have still to read, over the small inputs, over one another."""
    f = lib.rf_qk_norm_rope
    pages = dict(q_out=5 * 2048, k_out=160 * 512, v_out=160 * 512)        # bytes of each output
    for out in pages:
        for name in ("q", "k", "v", "positions", "freq", "slots", "qw"):
            assert f(*rope_args(**{name: at(20), out: at(20)})) == 1 or (out, name) == ("q_out", "q"), (out, name)
            assert f(*rope_args(**{name: at(20, pages[out] - 16), out: at(20)})) == 1, (out, name)
    assert f(*rope_args(q_out=at(7))) == 1                      # on k_out
    assert f(*rope_args(v_out=at(7, 160 * 512 - 16))) == 1
    assert f(*rope_args(v_out=at(7, 160 * 512))) == 4           # side by side: no device here, but not refused
    # without a cache; in place only where the rows lie one behind the other
    dense = dict(slots=NULL, v=NULL, v_out=NULL)
    assert f(*rope_args(**dense, q_out=at(0), q_step=1032)) == 1
    assert f(*rope_args(**dense, k_out=at(1), k_step=264)) == 1
    assert f(*rope_args(**dense, k_out=at(1, 16))) == 1
    assert f(*rope_args(**dense, q_out=at(0, 2048))) == 1       # a token on
    assert f(*rope_args(**dense, k_out=at(0), q_step=1280)) == 1
    # q, k and v beside one another in rows of 1544 values, an output over the last row's end
    assert f(*rope_args(**dense, k=at(0, 2048), q_step=1544, k_step=1544, k_out=at(0, 4 * 3088 + 2048 + 496))) == 1
    # the cache is not k's place
    assert f(*rope_args(k_out=at(1))) == 1


def test_python_layer_refuses_cpu_tensors_and_bad_shapes():
    import cascaded_reductions_gb300 as rf
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)                                   # noqa: E731
    q, k = torch.zeros(4, 8, 128, dtype=torch.bfloat16), torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    f = torch.ones(64)
    for call in (lambda: rf.page_tables(i(4), i(4), i(4, 3), i(9), i(1), 16, 8),
                 lambda: rf.qk_norm_rope(q, k, i(1, 4), f),
                 lambda: rf.qk_norm_rope(q, k, i(4), f),
                 lambda: rf.qk_norm_rope(q[0], k, i(1, 4), f),
                 lambda: rf.qk_norm_rope(q, k, i(1, 4), f, slots=i(4)),
                 lambda: rf.qk_norm_rope(q, k, i(1, 4), f, v=k)):
        with pytest.raises(ValueError):
            call()


def plan_args(**o):
    return [o.get("starts", at(0)), o.get("lens", at(1)), o.get("B", 4), o.get("T", 100), o.get("H", 8),
            o.get("Hkv", 2), o.get("max_new", 20), o.get("max_len", 1000), o.get("window", 0), o.get("sinks", 0),
            o.get("plan", at(2)), ctypes.c_size_t(o.get("bytes", 1 << 40)), NULL]


def attn_args(**o):
    return [o.get("q", at(0)), o.get("kp", at(1)), o.get("vp", at(2)), o.get("pages", 300), o.get("page", 16),
            o.get("table", at(3)), o.get("width", 64), o.get("plan", at(4)), ctypes.c_size_t(o.get("bytes", 1 << 40)),
            o.get("B", 4), o.get("T", 100), o.get("H", 8), o.get("Hkv", 2), o.get("D", 128), o.get("max_new", 20),
            o.get("max_len", 1000), o.get("window", 0), o.get("sinks", 0), F(o.get("scale", 0.1)), o.get("dtype", 1),
            o.get("out", at(5)), NULL, NULL]


@pytest.mark.parametrize("call,args", [("rf_paged_plan", plan_args), ("rf_attn_paged", attn_args)])
def test_paged_size_refusals(lib, call, args):
    f = getattr(lib, call)
    for name in ("B", "T", "H", "Hkv", "max_new", "max_len"):
        assert f(*args(**{name: 0})) == 1, name
        assert f(*args(**{name: -1})) == 1, name
    assert f(*args(H=7)) == 1                       # not a multiple of Hkv
    assert f(*args(max_new=101)) == 1               # more than there are rows
    assert f(*args(window=-1)) == 1
    assert f(*args(sinks=-1)) == 1
    assert f(*args(plan=NULL)) == 1
    big = (1 << 30) + 1
    assert f(*args(max_len=big, width=1 << 27)) == 2
    assert f(*args(T=1 << 28, H=8)) == 2
    assert f(*args(B=(1 << 20) + 1, width=64)) == 2
    assert f(*args(H=(1 << 16) + 2)) == 2
    assert f(*args(plan=at(4, 128))) == 3


def test_plan_refusals(lib):
    for name in ("starts", "lens"):
        assert lib.rf_paged_plan(*plan_args(**{name: NULL})) == 1, name
    lib.rf_paged_plan_bytes.restype = ctypes.c_size_t
    for bad in ((0, 1, 1, 1, 1, 1, 0, 0), (1, 1, 3, 2, 1, 1, 0, 0), (1, 1, 1, 1, 2, 1, 0, 0), (1, 1, 1, 1, 1, 1, -1, 0)):
        assert lib.rf_paged_plan_bytes(*bad) == 0


def test_plan_with_slots_refusals(lib):
    """As the plan without: the slots stand behind the lengths."""
    def f(slots=at(9), **o):
        a = plan_args(**o)
        return lib.rf_paged_plan_slots(*a[:2], slots, *a[2:])
    assert f(slots=NULL) == 1
    for name in ("starts", "lens", "plan"):
        assert f(**{name: NULL}) == 1, name
    for name in ("B", "T", "H", "Hkv", "max_new", "max_len"):
        assert f(**{name: 0}) == 1, name
    assert f(window=-1) == 1 and f(sinks=-1) == 1 and f(max_new=101) == 1
    assert f(max_len=(1 << 30) + 1) == 2
    assert f(plan=at(4, 128)) == 3


def test_attn_refusals(lib):
    f = lib.rf_attn_paged
    for name in ("q", "kp", "vp", "table", "out"):
        assert f(*attn_args(**{name: NULL})) == 1, name
    for name in ("pages", "page", "width", "D"):
        assert f(*attn_args(**{name: 0})) == 1, name
    assert f(*attn_args(width=62)) == 1             # 992 keys
    for scale in (float("nan"), float("inf")):
        assert f(*attn_args(scale=scale)) == 1
    assert f(*attn_args(dtype=3)) == 1
    assert f(*attn_args(dtype=0)) == 2              # fp32
    assert f(*attn_args(D=64)) == 2
    assert f(*attn_args(scale=0.0)) == 2
    assert f(*attn_args(scale=-0.1)) == 2
    for page in (1, 8, 24, 48, 512):
        assert f(*attn_args(page=page, width=2000)) == 2, page
    assert f(*attn_args(pages=1 << 30)) == 2
    assert f(*attn_args(width=1 << 30)) == 2
    for name in ("q", "kp", "vp", "out"):
        assert f(*attn_args(**{name: at(20, 8)})) == 3, name


def test_python_layer_of_the_paged_attention():
    import cascaded_reductions_gb300 as rf
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)                                   # noqa: E731
    q, kp = torch.zeros(4, 8, 128, dtype=torch.bfloat16), torch.zeros(9, 2, 16, 128, dtype=torch.bfloat16)
    plan = rf.PagedPlan(torch.zeros(100, dtype=torch.uint8), (0, 2, 4, 8, 2), 2, 48, 0, 0)
    for call in (lambda: rf.paged_plan(i(3), i(2), 4, 8, 2, 2, 48),
                 lambda: rf.attn_paged(q, kp, kp, i(2, 3), plan),
                 lambda: rf.attn_paged(q[0], kp, kp, i(2, 3), plan),
                 lambda: rf.attn_paged(q, kp, kp, i(6), plan)):
        with pytest.raises(ValueError):
            call()


def test_quick_calls_leave_what_they_cannot_take_to_python():
    import cascaded_reductions_gb300 as rf
    if rf._calls is None:
        pytest.skip("the extension is not built here")
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)                                   # noqa: E731
    q, k = torch.zeros(4, 8, 128, dtype=torch.bfloat16), torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    c = rf._calls
    assert c.page_tables(1, i(4), i(4), i(4, 3), i(9), i(1), 16, 8) is None             # not on a GPU
    assert c.page_tables(1, i(4), i(4), i(4, 3), i(9), i(1), 16) is None                # too few
    assert c.qk_norm_rope(1, q, k, i(1, 4), torch.ones(64), None, None, None, False, 1e-6, None, None, None,
                          None) is None
    assert c.qk_norm_rope(1, q, k, i(1, 4), torch.ones(64), None, None, None, 0, 1e-6, None, None, None,
                          None) is None                                                 # interleaved is no bool
    kp = torch.zeros(9, 2, 16, 128, dtype=torch.bfloat16)
    sizes = (0, 2, 4, 8, 2)
    assert c.attn_paged(1, q, kp, kp, i(2, 3), torch.zeros(9, dtype=torch.uint8), sizes, 2, 48, 0, 0, None) is None
    assert c.attn_paged("x", q, kp, kp, i(2, 3), None, sizes, 2, 48, 0, 0, None) is None


def test_kernels_that_divide_their_registers_have_them():
    """Read from the compiler's report of the library in place."""
    import glob
    import os

    from conftest import load_builder
    b = load_builder()
    b.build()
    want, seen = b.divided_registers(), {}
    for path in glob.glob(os.path.join(b.OBJDIR, "paged_*.ptxas")):
        with open(path) as f:
            seen.update(b.registers(f.read()))
    for part in ("paged_pair_kernel", "paged_decode_kernel"):
        mine = {n: r for n, r in seen.items() if part in n}
        assert len(mine) == 2 and set(mine.values()) == {want[part]}, (part, mine)


def test_other_registers_of_the_teams_kernel_are_told(capfd):
    from conftest import load_builder
    b = load_builder()
    report = ("ptxas info    : Compiling entry function '_Z19paged_decode_kernelI1P' for 'sm_103a'\n"
              "ptxas info    : Used {} registers, used 16 barriers\n")
    b._report_pairs(report.format(160))
    assert "RF_ERR_UNSUPPORTED" in capfd.readouterr().err
    b._report_pairs(report.format(b.divided_registers()["paged_decode_kernel"]))
    assert capfd.readouterr().err == ""
