"""ft_kv_append where several tokens share a block: every number of them with every remainder, and blocks whose tokens
belong to many sequences, empty ones between them."""
import pytest
import torch

from _kv import Cache
from test_gpu_kv_append import Step

pytestmark = pytest.mark.gpu


def lone():
    """Tokens that go one a block; 2 share one from twice as many on, 4 at most."""
    return 14 * torch.cuda.get_device_properties(0).multi_processor_count


def check_all(c, step):
    """q_out, the stored keys and values, weights and positions of every token, and that nothing else changed."""
    k0, v0, pos0, mass0 = c.k.clone(), c.v.clone(), c.pos.clone(), c.mass.clone()
    step.run()
    assert c.status.item() == 0
    t, b, slot = (torch.tensor(x, device="cuda") for x in zip(*step.slots()))
    page, s = c.table.long()[b, slot // c.page], slot % c.page
    # as in test_gpu_kv_append: bf16 rounds by 2^-8, sine, cosine and the rotation come to 2^-21 of the pair
    want, size = step.turned(step.q)
    assert ((step.q_out.double() - want).abs() <= want.abs() * 2.0 ** -8 + size * 2.0 ** -21)[t].all()
    left = torch.ones(step.T, dtype=torch.bool, device="cuda")
    left[t] = False
    assert (step.q_out[left] == 7.0).all()
    want, size = step.turned(step.k)
    got = c.k[page, :, s].double()
    assert ((got - want[t]).abs() <= want[t].abs() * 2.0 ** -8 + size[t] * 2.0 ** -21).all()
    assert torch.equal(c.v[page, :, s], step.v[t])
    assert (c.mass[page, :, s] == 0).all()
    assert torch.equal(c.pos[page, :, s], step.positions[0, t][:, None].expand(-1, c.kv_heads))
    for x, x0 in ((c.k.view(torch.int16), k0.view(torch.int16)), (c.v.view(torch.int16), v0.view(torch.int16)), (c.pos, pos0),
                  (c.mass.view(torch.int32), mass0.view(torch.int32))):
        x0[page, :, s] = x[page, :, s]
        assert torch.equal(x, x0)


@pytest.mark.parametrize("more", [-1, 0, 1, 2, 3])
@pytest.mark.parametrize("times", [1, 2, 3, 4])
def test_tokens_around_each_number_a_block_takes(times, more):
    T = times * lone() + more
    new = [T - 1030, 1, 0, 1029]
    c = Cache([n + 3 if n else 0 for n in new], 2, 1, 64, 64, seed=T)
    check_all(c, Step(c, new, 2))


@pytest.mark.parametrize("times", [2, 3, 5])
def test_blocks_of_tokens_of_many_sequences(times):
    """Prompts of 0 to 40 tokens: four tokens of a block can be of four sequences, with empty and idle ones between."""
    new, i = [], 0
    end = times * lone()
    while sum(new) < end:
        i += 1
        new.append([1, 0, 2, 1, 0, 0, 1, 3, 40, 0, 5, 1, 1, 1, 1][i % 15])
    lengths = [n + (j % 4) if n or j % 3 else 0 for j, n in enumerate(new)]
    c = Cache(lengths, 2, 1, 64, 8, seed=times)
    check_all(c, Step(c, new, 2, pad=7, seed=times))
