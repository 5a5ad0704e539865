"""CPU checks of the entry points of the 4-bit cache and of the rotation: bad arguments are
refused, with a reason, before anything touches CUDA, and numbers that a C int does not hold in
the binding."""
import ctypes

import pytest

CREATE4 = dict(blocks=16, n_pages=4, page_size=16, kv_heads=2, head_dim=64, q_heads=4, k_unit=0.5, v_unit=2.0, prompt_bytes=0)


@pytest.fixture(scope="module")
def lib():
    from heterogeneous_lora_gemm_gb300 import build as b
    b.build()
    from heterogeneous_lora_gemm_gb300 import mlora
    return mlora


@pytest.mark.parametrize("change,code", [
    (dict(blocks=None), 1), (dict(blocks=24), 1), (dict(n_pages=0), 1), (dict(kv_heads=0), 1), (dict(q_heads=0), 1),
    (dict(q_heads=5), 1), (dict(q_heads=65536), 1), (dict(k_unit=0.0), 1), (dict(k_unit=-1.0), 1),
    (dict(k_unit=float("nan")), 1), (dict(v_unit=float("inf")), 1), (dict(v_unit=2.0 ** 61), 1), (dict(v_unit=2.0 ** -61), 1),
    (dict(page_size=8), 8), (dict(page_size=24), 8), (dict(page_size=272), 8), (dict(head_dim=8), 8),
    (dict(head_dim=72), 8), (dict(head_dim=272), 8), (dict(n_pages=1 << 27), 8),
])
def test_create4_refuses(lib, change, code):
    h = ctypes.c_void_p(123)
    args = {**CREATE4, **change}
    assert lib.lib().mlora_cache_create4(*args.values(), ctypes.byref(h)) == code
    assert h.value is None and lib.last_error()
    assert lib.lib().mlora_cache_create4(*args.values(), None) == 1


@pytest.mark.parametrize("head_dim,rotary_dim,freq,code", [
    (64, 64, None, 1), (8, 0, None, 8), (72, 16, None, 8), (272, 16, None, 8), (64, 80, [0.0] * 40, 8), (64, -16, None, 8),
    (64, 24, [0.0] * 12, 8), (64, 16, [0.0] * 7 + [float("nan")], 1), (64, 16, [1025.0] + [0.0] * 7, 1),
])
def test_rotary_create_refuses(lib, head_dim, rotary_dim, freq, code):
    h = ctypes.c_void_p(123)
    table = (ctypes.c_double * len(freq))(*freq) if freq else None
    assert lib.lib().mlora_rotary_create(head_dim, rotary_dim, table, 0, ctypes.byref(h)) == code
    assert h.value is None and lib.last_error()
    assert lib.lib().mlora_rotary_create(head_dim, rotary_dim, table, 0, None) == 1


def test_null_rotary_is_invalid_arg(lib):
    L = lib.lib()
    assert L.mlora_rotary_apply(None, 16, 64, 64, 16, 64, 64, 1, 16, 64, 64, 16, 64, 64, 1, 1, 1, None, None, 0.0, None, 16,
                                1, 1, None) == 1
    assert L.mlora_rotary_status(None, None) == 1
    assert L.mlora_rotary_destroy(None) == 0


@pytest.mark.parametrize("number", [2 ** 31, 2 ** 32 + 5, -2 ** 32 + 5])
def test_functions_refuse_numbers_past_32_bits(lib, number, monkeypatch):
    class Untouched:
        def __getattr__(self, name):
            raise AssertionError(name)

    monkeypatch.setattr(lib, "_lib", Untouched())
    for name in ("n_pages", "page_size", "kv_heads", "head_dim", "q_heads"):
        make = {("blocks_ptr" if k == "blocks" else k): v for k, v in CREATE4.items()}
        with pytest.raises(ValueError):
            lib.mlora_cache_create4(**{**make, name: number})
    for size in (-1, 2 ** 64):
        with pytest.raises(ValueError):
            lib.mlora_cache_create4(**{**make, "prompt_bytes": size})
    with pytest.raises(ValueError):
        lib.mlora_rotary_create(number, 16, [0.0] * 8, False)
    with pytest.raises(ValueError):
        lib.mlora_rotary_create(64, 16, [0.0] * 7, False)
    call = dict(rotary=0, Q_ptr=16, q_row_stride=64, q_head_stride=64, Q_out_ptr=16, qo_row_stride=64, qo_head_stride=64,
                q_heads=1, K_ptr=16, k_row_stride=64, k_head_stride=64, K_out_ptr=16, ko_row_stride=64, ko_head_stride=64,
                kv_heads=1, dtype=1, T=1, q_weight_ptr=None, k_weight_ptr=None, eps=0.0, offsets_ptr=None, lengths_ptr=16,
                n_seqs=1, max_new=1, stream=0)
    for name in ("T", "n_seqs", "max_new", "q_heads", "kv_heads"):
        with pytest.raises(ValueError):
            lib.mlora_rotary_apply(**{**call, name: number})
