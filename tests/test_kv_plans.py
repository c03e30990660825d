"""How kv_attention plans prompts, on the host: nothing here reaches a HIP call.

The kernel of many rows holds 32 rows a wave.  A CU's LDS (160 KB) and registers hold so many of its workgroups:
two of four waves where the keys' and values' two stages (with remainders for fp16 and fp32 outputs) fit twice,
else one."""
import ctypes

import pytest

from tests.test_kv_options import option
from tests.test_serving_abi import cache, q  # noqa: F401

CUS = 256


def fit(dim, dt, waves):
    tokens = 32 if dt != 2 and dim > 128 else 64
    lds = 2 * tokens * dim * 2 * (2 if dt == 2 else 4)
    return 2 if waves == 4 and dim <= 128 and 2 * lds <= 160 * 1024 else 1


def plan(q, dim, hq, hkv, dt, batch, new, ctx, kernel=0, window=0):
    info, c = q.binding.KvPlanInfo(), cache(q, heads=hkv, dim=dim)
    assert q.lib().q4gsw_kv_attention_plan(ctypes.byref(c), batch, batch * new, hq, new, ctx, window, dt, option(q, kernel),
                                           ctypes.byref(info)) == 0
    return info


@pytest.mark.parametrize("dt", [0, 1, 2])
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
def test_splits_fill_the_gpu_once(q, dim, dt):  # noqa: F811
    """Keys are split only while all workgroups fit the GPU at once."""
    for hq, hkv in ((32, 8), (8, 1), (4, 4)):
        for batch in (1, 2, 3, 8, 40):
            for new in (40, 130, 700, 1024, 2048, 5000):
                for ctx in (new, new + 900, new + 7000, new + 60000):
                    for window in (0, 1000):
                        if new * hq // hkv <= 32:
                            continue
                        p = plan(q, dim, hq, hkv, dt, batch, new, ctx, 2, window)
                        groups = batch * hkv * -(-new * hq // hkv // (32 * p.waves))
                        assert p.waves in ((4, 8) if dim <= 128 else (4,))
                        assert p.splits == 1 or groups * p.splits <= CUS * fit(dim, dt, p.waves), (hq, batch, new, ctx, p.waves)


# us of the kernels of few and many rows, forced, one MI355X (fp32: as fp16 within 3%)
MEASURED = [
    # dim, hq, hkv, type, batch, new, ctx, few, many
    (128, 32, 8, 2, 1, 512, 512, 19.3, 22.7),
    (128, 32, 8, 2, 1, 2048, 2048, 118.0, 71.1),
    (128, 32, 8, 2, 1, 4096, 4096, 382.4, 164.8),
    (128, 32, 8, 1, 1, 1024, 8000, 372.4, 233.7),
    (128, 32, 8, 1, 2, 2048, 2048, 219.2, 137.2),
    (128, 32, 8, 2, 8, 40, 3000, 58.2, 44.4),
    (64, 32, 8, 1, 1, 1024, 1024, 27.0, 34.4),
    (64, 32, 8, 1, 2, 2048, 2048, 127.1, 82.1),
    (64, 32, 8, 1, 1, 4096, 4096, 222.0, 146.0),
    (64, 32, 8, 0, 1, 1024, 8000, 219.3, 148.7),
    (64, 32, 8, 2, 3, 700, 2500, 126.6, 76.1),
    (96, 32, 8, 1, 1, 1024, 8000, 298.6, 199.4),
    (192, 16, 4, 2, 1, 4096, 4096, 311.0, 202.5),
    (192, 16, 4, 1, 1, 2048, 16000, 943.2, 1149.3),
    (256, 16, 4, 2, 2, 2048, 2048, 235.2, 152.1),
    (256, 16, 4, 2, 1, 1024, 8000, 381.4, 252.4),
    (256, 16, 4, 1, 1, 2048, 2048, 130.4, 198.3),
    (256, 16, 4, 1, 3, 2048, 8192, 1734.7, 2026.0),
    (256, 16, 4, 0, 3, 2048, 8192, 1744.0, 2029.7),
    (128, 8, 1, 1, 1, 1024, 8000, 106.0, 77.8),
    (128, 8, 1, 1, 8, 40, 3000, 25.9, 33.0),
]


# drafts and short prompts: a turn of the kernel of many rows costs more than they have to do
SHORT = [
    (128, 8, 2, 2, 6, 14, 14, 7.5, 9.4),
    (96, 16, 4, 2, 1, 28, 28, 7.2, 8.5),
    (128, 32, 4, 1, 1, 21, 51, 7.7, 10.7),
    (256, 48, 8, 2, 2, 32, 32, 11.3, 16.2),
    (192, 6, 1, 1, 2, 38, 38, 9.3, 14.7),
    (64, 16, 4, 2, 7, 59, 59, 6.9, 8.1),
    (192, 16, 8, 1, 3, 47, 47, 9.6, 14.1),
    (64, 1, 1, 2, 2, 43, 51, 6.2, 7.2),
]
# windows: a workgroup sees the window and its own tokens, not all of the prompt's
WINDOWS = [
    (64, 32, 4, 2, 1, 2370, 2370, 48.7, 25.2, 421),
    (128, 32, 8, 2, 1, 1764, 3901, 47.7, 26.1, 224),
    (128, 8, 2, 2, 3, 1656, 1656, 32.0, 22.3, 180),
    (256, 64, 8, 1, 1, 1169, 1170, 116.4, 95.7, 183),
]


@pytest.mark.parametrize("case", MEASURED + SHORT + WINDOWS, ids=lambda c: "-".join(map(str, c[:7])))
def test_the_faster_kernel_is_taken(q, case):  # noqa: F811
    few, many, *window = case[7:]
    assert plan(q, *case[:7], 0, *window).kernel == (1 if few < many else 2)


@pytest.mark.parametrize("kernel", [1, 2])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_splits_of_a_window(q, dim, kernel):  # noqa: F811
    """Rows behind a window are split as the same rows behind that many keys, whatever the prompt's length."""
    for window, new, ctx in ((200, 3000, 20000), (500, 1000, 1000), (4096, 300, 60000)):
        p = plan(q, dim, 4, 1, 2, 1, new, ctx, kernel, window)
        blocks = (window + 64 * 4 + 62) // 32
        assert p.splits <= max(1, -(-blocks // (8 if kernel == 1 else 16))), (window, new, ctx)
