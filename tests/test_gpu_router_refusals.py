"""A router call that the library refuses says so, without room for its outputs first."""
import pytest

import bit_quantized_fine_amd as q
from gpu_util import dev, need_gpu, say, torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kw", [dict(topk=2 ** 31 - 1), dict(topk=65), dict(topk=0), dict(topk=-2 ** 31),
                                dict(topk=2, groups=3), dict(topk=2, groups=2 ** 31 - 1)])
def test_refused(kw):
    need_gpu()
    say(f"router, refused: {kw}")
    x = torch.zeros(4096, 128, device=dev())
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    with pytest.raises(q.QloraError):
        q.qlora_router_fwd(x, **kw)
    assert torch.cuda.max_memory_allocated() - before < 64 << 20
