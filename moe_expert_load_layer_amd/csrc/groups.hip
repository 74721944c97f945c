// Host side of groups.h.
#include "groups.h"

namespace ep {

bool layout_groups(const ep_layout_t *layout, int32_t groups, bool slots, GroupRows *where) {
    where->slot_home = where->slot_spare = nullptr;
    if (!layout) return true;
    if (!layout_ok(layout) || layout->num_phys != groups || (layout->num_spare > 0 && !slots)) return false;
    const Tables T = tables_of(*layout);
    where->slot_home = T.slot_home;
    where->slot_spare = T.slot_spare;
    return true;
}

}  // namespace ep
