"""The counters stored for the benchmark's dominant kernel are of the sources
as they are: after a change to any of them (headers they share with other
kernels among them) they are taken again, with the command that the file
holds, or the benchmark would report no traffic."""
import bench


def test_stored_traffic_is_of_the_present_sources():
    got = bench.measured_traffic()
    assert got is not None, "take %s again: a source of the kernel changed" % bench.TRAFFIC_FILE
    with open(bench.TRAFFIC_FILE) as f:
        kv = dict(line.strip().split(": ") for line in f if not line.startswith("#"))
    io = bench.DOMINANT_ITEMS_PER_LAUNCH * bench.KERNEL_IO_LIMBS["comb_ip"] * (1 << 16) * 8
    assert int(kv["kernel_io_bytes_per_launch"]) == io
    # each launch reads and writes every limb once; keys shared by a launch's items or lines fetched twice are the rest
    assert 0.9 * io < got < 1.2 * io
