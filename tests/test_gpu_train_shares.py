"""The experts' gradients of a share of the experts (expert-parallel), whose tiles
are chosen by the rows that an even routing keeps: shares of 1/4 to 1/16, evenly
routed and crowded far past that, with source blocks; and short segments of many
blocks, each of which fills a step."""
import pytest

import test_gpu_train as train

pytestmark = pytest.mark.gpu

SHARES = [dict(M=512, H=1024, F=512, E=16, k=8, held=2, base=7), dict(M=300, H=512, F=256, E=16, k=4, held=4, base=3),
          dict(M=700, H=256, F=512, E=64, k=8, held=8, base=56), dict(M=64, H=1088, F=704, E=64, k=8, held=8),
          dict(M=1000, H=256, F=512, E=128, k=8, held=8, base=60, S=4), dict(M=2000, H=512, F=1024, E=64, k=4, held=4, base=1),
          dict(M=2000, H=1088, F=704, E=16, k=2, held=2, base=5), dict(M=256, H=2048, F=1408, E=16, k=2, held=1, base=9),
          # most pairs of every token here: many times the rows that the tiles are chosen for
          dict(M=900, H=512, F=320, E=32, k=2, held=2, base=4, crowd=9.0), dict(M=3000, H=192, F=256, E=16, k=1, held=1, base=2, crowd=9.0),
          dict(M=400, H=1088, F=2112, E=16, k=1, held=1, base=0, crowd=9.0), dict(M=1200, H=320, F=448, E=64, k=3, held=4, base=8, crowd=9.0, S=3),
          # a share of which an even routing keeps no row
          dict(M=2, H=256, F=320, E=512, k=1, held=1, base=300, crowd=60.0),
          # no pair at all
          dict(M=40, H=256, F=320, E=8, k=2, held=2, base=3, skip=(3, 4))]


# short segments of many source blocks
BLOCKS = [dict(M=2048, H=256, F=512, E=16, k=1, S=32), dict(M=512, H=512, F=512, E=16, k=1, S=8), dict(M=600, H=320, F=448, E=4, k=2, S=64),
          dict(M=12000, H=256, F=320, E=8, k=1, S=8), dict(M=40, H=192, F=256, E=30, k=1, S=30), dict(M=700, H=1088, F=448, E=32, k=2, S=16, held=4, base=11)]

# few tiles of long reductions, which the kept products do not cut
LONG = [dict(M=600, H=3328, F=576, E=2, k=2, held=1), dict(M=1024, H=4096, F=512, E=8, k=1), dict(M=300, H=5824, F=192, E=20, k=3)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHARES + BLOCKS + LONG)
def test_experts_of_a_share(shape, dtype):
    train.test_experts(shape, dtype)
