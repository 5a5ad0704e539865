"""CPU checks of the binding of the 8-bit cache: a number that a C int does not hold is refused
(ctypes would pass its low 32 bits: a window of 2^32 + 5 as one of 5)."""
import pytest

torch = pytest.importorskip("torch")

from heterogeneous_lora_gemm_gb300 import Cache, mlora  # noqa: E402

TOO_MUCH = [2 ** 31, 2 ** 32, 2 ** 32 + 5, -2 ** 32 + 5]


class Recorder:
    """In the library's place: the arguments of each call."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *a: self.calls.append((name, a)) or 0


@pytest.fixture
def recorder(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(mlora, "_lib", r)
    return r


@pytest.fixture
def cache(recorder):
    c = Cache.__new__(Cache)
    c.handle, c._lib, c.device, c._index = None, recorder, torch.device("cpu"), -1
    c._dtypes, c._i32 = {torch.bfloat16: mlora.MLORA_BF16, torch.float32: mlora.MLORA_F32}, torch.int32
    c._raw_stream = lambda index: 0
    c.kv_heads, c.q_heads, c.page_size, c.head_dim = 2, 4, 16, 64
    return c


def step(T=3):
    return torch.zeros(T, dtype=torch.int32), torch.zeros((T, 2), dtype=torch.int32)


@pytest.mark.parametrize("number", TOO_MUCH)
def test_cache_refuses_numbers_past_32_bits(cache, recorder, number):
    k, q = torch.zeros((3, 2, 64)), torch.zeros((3, 4, 64))
    for call in (lambda: cache.append(k, k, *step(), max_new=number), lambda: cache.read(k, k, *step(), max_new=number),
                 lambda: cache.attend(q, q, *step(), max_new=number), lambda: cache.attend(q, q, *step(), window=number)):
        with pytest.raises(ValueError):
            call()
    assert not recorder.calls


def test_cache_refuses_rows_past_32_bits(cache, recorder):
    k = torch.zeros((1, 2, 64)).expand(2 ** 32 + 1, 2, 64)
    with pytest.raises(ValueError):
        cache.append(k, k, *step(1), offsets=torch.zeros(2, dtype=torch.int32))
    assert not recorder.calls


def test_cache_passes_numbers_of_32_bits_on(cache, recorder):
    q = torch.zeros((3, 4, 64))
    cache.attend(q, q, *step(), max_new=2 ** 31 - 1, window=2 ** 31 - 1, scale=0.5)
    cache.attend(q, q, *step(), max_new=-1, window=-1)       # (the library's to refuse)
    (name, first), (_, second) = recorder.calls
    assert name == "mlora_cache_attend" and first[14:17] == (2 ** 31 - 1, 0.5, 2 ** 31 - 1)
    assert second[14] == -1 and second[16] == -1


@pytest.mark.parametrize("number", TOO_MUCH)
def test_functions_refuse_numbers_past_32_bits(recorder, number):
    rows = dict(K_ptr=16, k_row_stride=128, k_head_stride=64, V_ptr=16, v_row_stride=128, v_head_stride=64)
    queries = dict(Q_ptr=16, q_row_stride=128, q_head_stride=64, O_ptr=16, o_row_stride=128, o_head_stride=64)
    rest = dict(cache=0, dtype=1, T=1, offsets_ptr=None, lengths_ptr=16, pages_ptr=16, n_seqs=1, width=1, max_new=1,
                stream=0)
    for name in ("T", "n_seqs", "width", "max_new"):
        for f, x in ((mlora.mlora_cache_append, rows), (mlora.mlora_cache_read, rows),
                     (mlora.mlora_cache_attend, {**queries, "scale": 1.0, "window": 0})):
            with pytest.raises(ValueError):
                f(**{**x, **rest, name: number})
    with pytest.raises(ValueError):
        mlora.mlora_cache_attend(**queries, **rest, scale=1.0, window=number)
    make = dict(k_codes_ptr=16, k_scale_ptr=16, v_codes_ptr=16, v_scale_ptr=16, n_pages=4, page_size=16, kv_heads=2,
                head_dim=64, q_heads=4, prompt_bytes=0)
    for name in ("n_pages", "page_size", "kv_heads", "head_dim", "q_heads"):
        with pytest.raises(ValueError):
            mlora.mlora_cache_create(**{**make, name: number})
    for size in (-1, 2 ** 64):
        with pytest.raises(ValueError):
            mlora.mlora_cache_create(**{**make, "prompt_bytes": size})
    assert not recorder.calls
