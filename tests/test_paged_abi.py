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
