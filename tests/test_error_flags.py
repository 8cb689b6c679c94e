"""The device error flags are read in one way, on the host and without a GPU."""
import glob
import os

from test_host_setup import CSRC, run_check


def test_a_flag_that_is_not_set_is_not_written(tmp_path):
    run_check("error_flag_check", tmp_path)


def test_flags_are_taken_by_that_alone():
    for path in glob.glob(os.path.join(CSRC, "*")):
        if os.path.basename(path) != "error_flag.h":
            assert "cudaMemcpyToSymbol" not in open(path).read(), path
