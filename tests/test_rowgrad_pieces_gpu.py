"""The gather's gradient around the sizes at which its pieces change, with runs of equal tokens that
end at, cross and fill pieces."""
import pytest
import torch

import embedding_table_gather_amd as etg
from tests import training_oracle as to
from tests.gpu_util import note

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [8, 9, 15, 16, 17, 129, 1023, 1024, 1025, 1040, 2049, 4095])
@pytest.mark.parametrize("length", [1, 7, 8, 9, 16, 40, 300])
def test_runs_and_pieces(n, length):
    # runs of `length` equal tokens, shuffled; every 11th id is bad
    V, d = 600, 72
    note(f"{n} ids in runs of {length}")
    gen = torch.Generator().manual_seed(n + length)
    ids = (torch.arange(n) // length * 37) % V
    ids[::11] = -1
    ids = ids[torch.randperm(n, generator=gen)].to(torch.int32).cuda()
    grad = torch.randn((n, d), generator=gen).cuda()
    old = torch.randn((V, d), generator=gen).to(torch.bfloat16).cuda()
    t = etg.Table(torch.zeros((V, d), dtype=torch.bfloat16, device="cuda"), etg.BF16, V, d)
    got = t.embed_gather_grad(grad, ids, scale=2.5, out_dtype=torch.float32)
    added = t.embed_gather_grad(grad, ids, scale=2.5, out=old.clone(), accumulate=True)
    torch.cuda.synchronize()
    to.check(got, *to.gather_grad(grad, ids, V, 2.5, torch.float32), "rows")
    to.check(added, *to.gather_grad(grad, ids, V, 2.5, torch.bfloat16, old), "rows, added")
