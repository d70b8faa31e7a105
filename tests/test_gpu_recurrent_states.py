"""What the state-space scan keeps of its states on the GPU: the same for every call that wants
the outputs, all bits of what a token adds, no error that grows with the length."""
import pytest
import torch

import chunked_gated_delta_11_gb300 as kda
import recurrent_ref as ref
from test_gpu_recurrent import cu_of, dev, gen, randn, run_ssm, ssm_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    kda.build.build()
    kda.load()


@pytest.mark.parametrize("lengths,H,G,P,S", [([300, 7, 0, 128], 3, 1, 64, 128), ([500], 2, 2, 128, 64), ([2300], 2, 1, 64, 128)])
def test_outputs_do_not_depend_on_who_wants_the_states(lengths, H, G, P, S):
    case = ssm_case(70, lengths, H, G, P, S, state=None, rate=0.5)
    out, fin = run_ssm("kda_ssm_fwd", case, lengths)
    alone, none = run_ssm("kda_ssm_fwd", case, lengths, output_final_state=False)
    half, fin16 = run_ssm("kda_ssm_fwd", case, lengths,
                          final_state=torch.empty((len(lengths), H, P, S), dtype=torch.bfloat16, device="cuda"))
    assert none is None
    assert torch.equal(out, alone) and torch.equal(out, half)
    assert torch.equal(fin.to(torch.bfloat16), fin16)
