"""GPU: groups of more than eight query heads (several units a KV head) with block tables on both sides of the
width from which the decode kernel takes the own tokens.  Tolerance as in test_gpu_prefix.py."""
import pytest

from tests.test_gpu_prefix import build, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,bk,bv", [("bf16", 4, 4), ("k8v4", 8, 4), ("packed", 4, 4), ("packed", 3, 2)])
@pytest.mark.parametrize("width", [120, 140, 300])
@pytest.mark.parametrize("hq,hkv", [(12, 1), (17, 1), (24, 2), (96, 8)])
def test_large_groups_with_wide_tables(cuda, tqlib, fmt, bk, bv, width, hq, hkv):
    case = build(cuda, tqlib, fmt, bk, bv, B=3, hq=hq, hkv=hkv, P=150, lens=[16 * width - 3, 20, 0], seed=width, width=width)
    check(cuda, tqlib, case, 150)
