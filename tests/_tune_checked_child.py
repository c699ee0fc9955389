"""Child process of tests/test_gpu_tune_checked.py: runs the shared cases with the library that
LP_LIBRARY names and saves the outputs, the backend id and the check word."""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

from invariant_token_logprobs_gb300 import lp, tune  # noqa: E402
from _tune_checked_cases import run_cases  # noqa: E402

lp.load(build_if_needed=False)
out = run_cases(tune)
torch.save({"out": out, "backend": lp.lp_backend_id(), "word": lp.lp_get_check_word()}, sys.argv[1])
