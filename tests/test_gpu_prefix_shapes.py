"""kvq_paged_prefix_attention at every number of query heads a KV head (1 to 8) and at head counts that leave the decode
kernel's head groups uneven, with groups whose rows cross a block of 128.  Tolerance: the decode tests' (harness.bound)."""
import dataclasses

import pytest

from quantized_paged_kv_gb300 import workloads as W
from tests import harness as H
from tests.test_gpu_prefix import _Call, _share

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    H.ensure_built()


@pytest.mark.parametrize("fmt", ["int8", "nvfp4", "bf16"])
@pytest.mark.parametrize("out_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 3])
@pytest.mark.parametrize("shape", [(1, 1, 128), (5, 2, 256), (6, 3, 128), (9, 4, 256), (1, 5, 128), (2, 6, 128),
                                   (4, 7, 128), (2, 8, 256), (3, 1, 256)])
def test_head_counts(shape, T, out_dtype, fmt):
    """Two groups and a lone sequence; the first group's rows (sequence, token, head) fill a block of 128 and part of
    another, with a sequence on the border."""
    Hkv, G, D = shape
    n = 130 // (G * T) + 2
    lens = [80 + 3 * (i % 9) for i in range(n)] + [60 + i for i in range(3)] + [33]
    offsets, pl = [0, n, n + 3], [80, 48]
    wl = _share(W.make("serving_int8", lens=("list", lens), seed=103), offsets, pl)
    wl = dataclasses.replace(wl, Hkv=Hkv, Hq=Hkv * G, D=D)
    gs = H.global_scales(wl, fmt)
    c = _Call(wl, fmt, offsets, pl, T=T, splits=2, out_dtype=out_dtype, gs=gs)
    c.launch(checked=True)
    border = 128 // (G * T)
    c.check(units=[(b, i, h) for b in {0, 1, border - 1, border, border + 1, n - 1, n, n + 2, n + 3} for i in range(T)
                   for h in sorted({0, Hkv // 2, Hkv - 1})])


def test_the_largest_launch():
    """4,096 launch sequences, the most that a device plan takes, in 500 groups and 24 lone sequences."""
    lens = [17 + b % 40 for b in range(1024)]
    offsets = [2 * g for g in range(501)]
    wl = _share(W.make("serving_int8", lens=("list", lens), seed=104), offsets, [16] * 500)
    wl = dataclasses.replace(wl, Hkv=1, Hq=3)
    c = _Call(wl, "int8", offsets, [16] * 500, T=4, splits=1)
    assert c.plan.batch == 4096
    c.launch(checked=True)
    c.check(units=[(b, i, 0) for b in (0, 1, 2, 511, 998, 999, 1000, 1001, 1023) for i in (0, 3)])
