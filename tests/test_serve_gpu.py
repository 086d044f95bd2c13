"""The serving layer (serve.py): prompts, forks and decode steps through the operators together (GPU)."""
import torch
import pytest

from gdn_chunkwise_ut_gb300 import device_status
from gdn_chunkwise_ut_gb300.serve import GdnLayer, main

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_decode_carries_a_prompt_on():
    """Two prompts of 100 and 37 tokens, then 30 more tokens each: as one longer prompt, and as decode
    steps behind the shorter one.  The two differ by the chunked rule's bf16 products (its o is within
    1e-2 of exact, relative Frobenius) and the projections' bf16 roundings behind it."""
    layer = GdnLayer(512, 2, 4, seed=1)
    pool = layer.pool(6)
    lengths, more = (100, 37), 30
    gen = torch.Generator(device=DEV)
    gen.manual_seed(2)
    x = [torch.randn((n + more, 512), generator=gen, device=DEV).to(torch.bfloat16) for n in lengths]

    def pack(parts):
        cu = torch.tensor([0, *torch.tensor([p.shape[0] for p in parts]).cumsum(0)], dtype=torch.int32, device=DEV)
        return torch.cat(parts)[None], cu

    whole, cu = pack(x)
    want, _ = layer.prefill(whole, torch.zeros_like(whole), pool, pool.index(pool.alloc(2)), cu)
    want = [want[0, cu[i]:cu[i + 1]][lengths[i]:] for i in range(2)]
    start, cu = pack([p[:n] for p, n in zip(x, lengths)])
    slots = pool.alloc(2)
    layer.prefill(start, torch.zeros_like(start), pool, pool.index(slots), cu)
    fork = pool.fork(slots[0])
    index = pool.index([slots[0], slots[1], fork[0]])
    out = []
    for t in range(more):
        tok = torch.stack([x[0][lengths[0] + t], x[1][lengths[1] + t], x[0][lengths[0] + t]])[:, None]
        out.append(layer.decode(tok, torch.zeros_like(tok), pool, index)[0][:, 0])
    got = torch.stack(out, 1)
    torch.cuda.synchronize()
    assert device_status() == 0
    assert torch.equal(got[0], got[2])  # the fork goes the way of its source
    for i in range(2):
        a, b = got[i].double(), want[i].double()
        assert ((a - b).norm() / b.norm()).item() <= 2e-2


def test_the_command_runs(monkeypatch, capsys):
    monkeypatch.setattr("sys.argv", ["serve", "--prompts", "2", "--samples", "2", "--tokens", "70", "--steps", "3"])
    main()
    assert "us a decode step" in capsys.readouterr().out
    assert device_status() == 0
