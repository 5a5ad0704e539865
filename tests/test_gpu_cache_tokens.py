"""Which tokens the attention over the 8-bit cache sums, to the token.  All scores are equal, and
token t's value is 127 in element t mod D and 0 elsewhere: output d of a row is then the number
of tokens t = d (mod D) that it sees, times 127 value scales (2^-7 here), over the number that it
sees.

Tolerance.  The weights are one number of at most 8 bits (2^-7 in the exponent's place, all of a
row alike), so that sums of up to 127 x 128 of them are exact in 24 bits, and so is the weights'
sum: what rounds is 1 / sum, the product with it (2^-24 each, twice for joined parts) and the
output, 2^-9 for bf16: within 2^-8 and 2^-20.  A token that is left out or taken twice moves a
count of at most 128 by one, that is by 2^-7 or more."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():   # pragma: no cover - CPU machine
    pytest.skip("needs a GPU", allow_module_level=True)

from heterogeneous_lora_gemm_gb300 import Cache, mlora  # noqa: E402
from test_gpu_cache import ATTENDS, F, TDT, Setup, offsets_of  # noqa: E402

# rows, lengths, H, G, D, page, window
PARTS = [     # the long axis is cut: few rows, and prompts of few row tiles
    ([1], [8000], 1, 2, 64, 16, 0), ([1], [20000], 2, 8, 256, 128, 0), ([2, 1], [9000, 17], 1, 4, 128, 64, 0),
    ([4], [6000], 1, 4, 80, 48, 0), ([1], [16000], 1, 4, 128, 64, 12345),
    ([20], [3000], 1, 1, 128, 64, 0), ([40, 3], [2000, 700], 1, 4, 64, 16, 0), ([20, 20, 1], [1100, 20, 0], 2, 2, 256, 32, 0),
    ([300], [2000], 1, 1, 256, 128, 500), ([5], [5000], 1, 8, 192, 48, 0), ([70], [4500], 1, 2, 80, 64, 3000),
    ([33], [40], 1, 1, 160, 16, 0), ([130], [8192], 1, 2, 64, 32, 0), ([17], [16000], 2, 2, 128, 128, 0),
]
AHEAD = [     # prompts converted ahead (more than 12 row tiles)
    ([250, 60, 410], [250, 500, 700], 1, 16, 128, 64, 0), ([250, 60, 410], [250, 500, 700], 1, 16, 80, 48, 150),
    ([900, 20], [1000, 300], 1, 8, 256, 32, 0), ([230, 1, 0], [3000, 900, 40], 1, 16, 64, 16, 1000),
]
WINDOWS = [(rows, lengths, 1, G, 64, ps, w)
           for rows, lengths, G in (([1, 2], [300, 131], 3), ([9, 20], [300, 131], 1), ([70, 40], [700, 131], 2))
           for ps in (16, 64) for w in (1, 2, 16, 17, 63, 64, 65, 128, 129)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,lengths,H,G,D,ps,window", ATTENDS + PARTS + AHEAD + WINDOWS)
def test_every_token_counts_once(rows, lengths, H, G, D, ps, window, dtype):
    assert max(lengths) <= 128 * D
    u = Setup(lengths, H, D, ps, Hq=H * G, seed=60)
    u.vc[:] = 0
    for t, n in zip(u.table, lengths):
        at = np.arange(max(n, 0))
        u.vc[t[at // ps], :, at % ps, at % D] = 127
    u.vs = np.where(np.isnan(u.vs), u.vs, F(2.0 ** -7))
    u.upload()
    Q = torch.zeros((sum(rows), H * G, D), dtype=TDT[dtype], device="cuda")
    pos = np.concatenate([np.arange(n - r, n) for r, n in zip(rows, lengths)])[:, None]
    lo = np.maximum(pos - window + 1, 0) if window else np.zeros_like(pos)
    d = np.arange(D)[None]
    want = ((pos - d) // D - (lo - 1 - d) // D) * 127 * 2.0 ** -7 / np.maximum(pos - lo + 1, 1)
    want[pos[:, 0] < 0] = 0.0
    for room in (256 << 20, 0):
        cache = Cache(*u.dev, H * G, prompt_bytes=room)
        O = torch.full_like(Q, float("nan"))
        cache.attend(Q, O, u.len, u.pages, offsets=offsets_of(rows), max_new=max(rows), window=window)
        got = O.double().cpu().numpy()
        off = np.abs(got - want[:, None]) > want[:, None] * (2.0 ** -8 if dtype == "bf16" else 2.0 ** -20)
        assert not (off | np.isnan(got)).any(), f"{off.sum()} of {off.size} off, first {np.argwhere(off | np.isnan(got))[0]}"
        assert cache.status() == mlora.MLORA_OK
