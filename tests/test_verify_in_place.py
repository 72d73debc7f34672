"""fk_verify does not write over the drafts it reads, on the CPU: a wave would read
what another had written."""
import struct

import exact_lloyd_means_amd as fk

VERIFY, FAKE = struct.Struct("@qqqPPPPqqiiPPPPPP"), 0x10000


def test_emitted_is_not_tokens():
    for accept, pick in ((FAKE, FAKE), (0, 0)):
        # tokens and emitted at one address; everything else is right
        args = VERIFY.pack(2, 5, 100, FAKE, 2 * FAKE, FAKE, 0, 100, 0, fk.FK_F32, 0, accept, pick, 0, FAKE, 2 * FAKE, 0)
        assert fk.lib.fk_verify(args, FAKE, 1 << 40, None) == fk.FK_EINVAL
        assert "emitted" in fk.lib.fk_last_error().decode()
