"""What lies behind a sequence's last token, more than a chunk of it: no row of y is
written there, and none of the inputs read, on every way a prompt can take."""
import pytest
import torch

from tests import gpu_util as gu
from tests.test_gpu_delta import Prompts
from tests.test_gpu_delta_parts import WAYS

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("way", range(len(WAYS)))
def test_rows_behind_the_last_sequence(io, way):
    """(the checks of Prompts: rows of no sequence hold NaN in the inputs, and 7 in y before and after)"""
    lens, H, G, P, N = WAYS[way]
    for last in (1, 8, 16, 17, 33, 48, 49, 64, 65, 128):
        gu.note(f"delta_scan, last of {len(lens)} has {last} tokens, H={H} P={P} N={N} {io}")
        p = Prompts([*lens[:-1], last], H, G, P, N, io, first=70, extra=140, seed=last)
        p.run()
        torch.cuda.synchronize()
        p.check([len(lens) - 1])
