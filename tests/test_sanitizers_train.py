"""The host side of the training entry points (argument checks, descriptor
batches, workspace sizes) under AddressSanitizer and UndefinedBehaviorSanitizer:
the library is rebuilt with both on its host pass and the host tests run
through it in a child process."""
import os

import pytest

from test_sanitizers import ROOT, _run


def test_training_host_checks_under_address_and_ub_sanitizers(tmp_path):
    from combine_router_top_expert_amd import build
    if not os.path.exists(build.HIPCC):
        pytest.skip("hipcc not present")
    lib = build.build(out=str(tmp_path / "libmok_san.so"), sanitize=True)
    _run({"LD_PRELOAD": build.sanitizer_runtime(), "MOK_LIB": lib},
         ["-m", "pytest", "-q", "-x", "-p", "no:cacheprovider",
          os.path.join(ROOT, "tests", "test_train_abi.py")])
