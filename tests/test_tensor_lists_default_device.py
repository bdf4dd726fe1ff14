"""Lists of tensors under a default device: the table is written by the host,
wherever torch puts new tensors."""
import pytest
import torch

from gpu_common import need_gpu, say


def test_table_is_built_in_host_memory():
    """Without a GPU the table is built and only then a device is missing;
    memory of the default device could not have been written."""
    import gram_newton_schulz_amd as gns
    if torch.cuda.is_available():
        pytest.skip("covered by the test below")
    with torch.device("meta"):
        with pytest.raises(RuntimeError) as e:
            gns.tensor_list([])
    assert not isinstance(e.value, gns.GnsError)


@pytest.mark.gpu
def test_default_device_is_the_gpu():
    gns = need_gpu()
    say("default device")
    with torch.device("cuda"):
        empty = gns.grad_norm([], max_norm=1.0)
        got = gns.clip_grad_norm_([torch.full((300, 3), 2.0)], 1.0, inv_scale=torch.tensor(0.5))
        state = [[torch.ones(70)] for _ in range(4)]
        gns.adamw_step(gns.adamw_list(*state), 1, lr=0.5, weight_decay=0.0)
    assert float(empty.norm) == 0.0 and float(got.norm) == 30.0
    # m = 0.9 + 0.1, v = 0.999 + 0.001: both corrected by their own 1 - beta
    assert torch.allclose(state[0][0], torch.full((70,), 1.0 - 0.5 * (1 / 0.1) / (1 / 0.001) ** 0.5, device="cuda"),
                          rtol=0, atol=1e-5)
